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
// Codes lie 6 to 12 % apart, and step t moves a moment by about 1 / t of itself, later by 1 - beta. Rounded to the nearest
// code a moment stands still once that is less than half the distance. So only the first SS1_ADAMW_NEAREST
// steps take the nearest code; a later one takes either neighbour, the farther one as often as the value lies towards
// it: the held value then follows the moment on average. What decides is a hash of step and element, so a step repeated
// gives the same bits. 2000 steps at the default betas, constant / normal gradients: r.m.s. update 1.01 / 1.02 of float32
// moments' (always nearest: 5.1 / 2.3, the held root 0.12 / 0.39 of the true one). Nearest up to 10 steps: held roots 0.98 to
// 1.04 of the true ones, spread 0.07 at most, as with either neighbour from the start; up to 16: 0.85.
//
// Memory-bound: bf16 weights with a float32 master copy move 28 bytes an element with float32
// moments, 16 with 8-bit ones. Every float32 operation is rounded on its own (no fused multiply-
// add), so that the codes are those of the same formula written with elementwise operations.
//
// 30 M bf16 weights with master copies: float32 moments 135 us (840 MB at 6.2 TB/s, 0.95 of the copy rate); 8 bits 93 us
// while codes are the nearest (482 MB, 5.2 TB/s, 0.79), where the issue slots of each element's root and quotient (57 %
// busy) and the loads that 64 registers a thread keep in flight bound it together, and 115 us past that (4.2 TB/s, 0.64),
// where random bits and neighbours add to the issue slots. Each rounding has a loop of its own: one loop with the
// choice inside took 40 % longer for both.
#include "ss1_ops.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <math.h>
#include <stdlib.h>

#include <algorithm>

namespace ss1 {
namespace {

using namespace op;

constexpr int kBlock = 256;              // elements of one scale: one warp, eight a lane
constexpr int kWarps = 8;
constexpr int kChunk = kBlock * kWarps * 4;   // elements of a CTA: four blocks a warp
constexpr int64_t kNearest = SS1_ADAMW_NEAREST;

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

// a * b rounded by itself: with `none` = -0, a * b + none has its value and its sign. `none` is a kernel
// parameter, because the assembler turns a constant -0 back into a product and joins that with the
// sum that follows.
__device__ __forceinline__ F2 times(F2 a, F2 b, F2 none) { return fma2(a, b, none); }

// Eight elements at `p`. WHOLE: all inside the tensor and on vector boundaries; else the first `n`, one at a
// time (0 in the others).
template <typename T, bool WHOLE>
__device__ __forceinline__ void load8(const T* p, int n, F2 (&f)[4]) {
    if (WHOLE) {
        Raw8<T> r;
        r.load_once(p);
        r.get(f);
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f(p[i]) : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = F2::of(v[2 * i], v[2 * i + 1]);
    }
}

template <typename T, bool WHOLE>
__device__ __forceinline__ void store8(T* p, int n, const F2 (&f)[4]) {
    if (WHOLE) {
        Raw8<T> r;
        r.set(f);
        r.store(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f<T>(i % 2 ? f[i / 2].hi() : f[i / 2].lo());
    }
}

template <bool WHOLE>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int n) {
    if (WHOLE) return __ldcs(reinterpret_cast<const uint2*>(p));
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
    return make_uint2(w[0], w[1]);
}

template <bool WHOLE>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint2 c) {
    if (WHOLE) {
        *reinterpret_cast<uint2*>(p) = c;
        return;
    }
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
}

__device__ __forceinline__ void decode8(uint2 c, float scale, F2 (&f)[4]) {
    const uint32_t w[2] = {c.x, c.y};
    const F2 by = F2::both(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i % 2)));
        const float2 x = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
        f[i] = F2::of(x.x, x.y) * by;
    }
}

// The block's scale from its largest magnitude over the warp; a NaN does not count.
__device__ __forceinline__ float block_scale(const F2 (&f)[4]) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) most = fmaxf(most, fmaxf(fabsf(f[i].lo()), fabsf(f[i].hi())));
    // magnitudes order like their bits: top = 1.f * 2^ex, and 448 is 1.75 * 2^8
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
    const int ex = (int)(top >> 23) - 127;
    const int e = (top & 0x7FFFFFu) <= 0x600000u ? ex - 8 : ex - 7;
    return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

// Random bits: two rounds of xor-shift and product (odd constants, from the golden ratio and the root of 3) on the lane's
// number in the tensor, by a key of the step; a linear congruence leads through the lane's eight elements.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ x >> 16) * 0x9E3779B9u;
    x = (x ^ x >> 15) * 0xBB67AE85u;
    return x ^ x >> 16;
}
__device__ __forceinline__ uint32_t step_key(int64_t step) {
    return mix((uint32_t)step * 0x9E3779B9u + (uint32_t)(step >> 32) * 0xBB67AE85u + 0x3C6EF373u);
}
__device__ __forceinline__ uint32_t lane_bits(uint32_t key, int64_t number) {
    return mix((uint32_t)number ^ (key + (uint32_t)(number >> 32) * 0x9E3779B9u));
}
__device__ __forceinline__ uint32_t next_bits(uint32_t x) { return x * 0xB7E15165u + 0x243F6A89u; }

// One of the two E4M3 values around x, |x| <= 448: the one away from 0 for as many of the 2^20 values of `bits` as x lies of the
// 2^20 parts of the way towards it. A code keeps a float's upper 3 bits of fraction, so the other 20 plus `bits`
// carry into them that often. Below 2^-6 codes lie 2^-9 apart, as they do from there to 2^-5.
__device__ __forceinline__ float neighbour(float x, uint32_t bits) {
    const float shift = fabsf(x) < 0x1p-6f ? copysignf(0x1p-6f, x) : 0.0f;
    const float y = __uint_as_float((__float_as_uint(x + shift) + bits) & 0xFFF00000u) - shift;
    return x == x ? y : x;
}

// The nearest codes, or (DITHER) neighbours by the upper 20 bits of each element's random word times TURN.
template <bool DITHER, uint32_t TURN>
__device__ __forceinline__ uint2 encode8(const F2 (&f)[4], float scale, uint32_t bits) {
    // 1 / scale, exactly: scale = 2^e with -126 <= e <= 121
    const F2 by = F2::both(__uint_as_float((254u << 23) - __float_as_uint(scale)));
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        F2 x = f[i] * by;   // exact but for results below 2^-126
        if (DITHER) {
            const uint32_t second = next_bits(bits);
            x = F2::of(neighbour(x.lo(), bits * TURN >> 12), neighbour(x.hi(), second * TURN >> 12));
            bits = next_bits(second);
        }
        w[i / 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x.lo(), x.hi()), __NV_SATFINITE, __NV_E4M3) << (16 * (i % 2));
    }
    return make_uint2(w[0], w[1]);
}

// Eight elements of one lane: `at` in the tensor, `block` their block, whose 32 lanes come here together.
template <int BITS, bool DITHER, bool WHOLE>
__device__ __forceinline__ void update8(const Entry& t, uint32_t flags, const Factors& f, F2 none, uint32_t key, int64_t at, int n,
                                        int64_t block, int lane) {
    F2 g[4], p[4], m[4], v[4], root[4];
    uint2 mc, vc;
    float ms, vs;
    if (flags & kGradBf16) load8<__nv_bfloat16, WHOLE>((const __nv_bfloat16*)t.g + at, n, g);
    else load8<float, WHOLE>((const float*)t.g + at, n, g);
    if (t.master) load8<float, WHOLE>(t.master + at, n, p);
    else if (flags & kParamBf16) load8<__nv_bfloat16, WHOLE>((const __nv_bfloat16*)t.p + at, n, p);
    else load8<float, WHOLE>((const float*)t.p + at, n, p);
    if (BITS == 32) {
        load8<float, WHOLE>((const float*)t.m + at, n, m);
        load8<float, WHOLE>((const float*)t.v + at, n, v);
    } else {
        mc = load_codes<WHOLE>((const uint8_t*)t.m + at, n);
        vc = load_codes<WHOLE>((const uint8_t*)t.v + at, n);
        ms = t.m_scale[block];
        vs = t.v_scale[block];
        decode8(mc, ms, m);
        decode8(vc, vs, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = times(v[i], v[i], none);
    }
    const F2 beta1 = F2::both(f.beta1), rest1 = F2::both(f.rest1), beta2 = F2::both(f.beta2), rest2 = F2::both(f.rest2);
    const F2 scale = F2::both(f.grad), eps = F2::both(f.eps), by_root = F2::both(f.root), keep = F2::both(f.keep), back = F2::both(-f.step);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const F2 gi = times(g[i], scale, none);
        m[i] = times(m[i], beta1, none) + times(gi, rest1, none);
        v[i] = times(v[i], beta2, none) + times(times(gi, gi, none), rest2, none);
        root[i] = F2::of(__fsqrt_rn(v[i].lo()), __fsqrt_rn(v[i].hi()));
        const F2 den = times(root[i], by_root, none) + eps;
        const F2 q = F2::of(__fdiv_rn(m[i].lo(), den.lo()), __fdiv_rn(m[i].hi(), den.hi()));
        p[i] = times(p[i], keep, none) + times(q, back, none);     // a - b is a + (-b)
    }
    if (t.master) store8<float, WHOLE>(t.master + at, n, p);
    if (flags & kParamBf16) store8<__nv_bfloat16, WHOLE>((__nv_bfloat16*)t.p + at, n, p);
    else store8<float, WHOLE>((float*)t.p + at, n, p);
    if (BITS == 32) {
        store8<float, WHOLE>((float*)t.m + at, n, m);
        store8<float, WHOLE>((float*)t.v + at, n, v);
        return;
    }
    if (!WHOLE) {   // what lies behind the tensor's end takes no part in the block's maximum
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = F2::of(2 * i < n ? m[i].lo() : 0.0f, 2 * i + 1 < n ? m[i].hi() : 0.0f);
            root[i] = F2::of(2 * i < n ? root[i].lo() : 0.0f, 2 * i + 1 < n ? root[i].hi() : 0.0f);
        }
    }
    ms = block_scale(m);
    vs = block_scale(root);
    const uint32_t bits = lane_bits(key, block * 32 + lane);
    mc = encode8<DITHER, 0xBB67AE85u>(m, ms, bits);
    vc = encode8<DITHER, 1>(root, vs, bits);
    // a positive root that rounded to code 0 takes code 1; most words have no zero byte
    uint32_t w[2] = {vc.x, vc.y};
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if ((w[h] - 0x01010101u) & ~w[h] & 0x80808080u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float r = i % 2 ? root[2 * h + i / 2].hi() : root[2 * h + i / 2].lo();
                if (r > 0.0f && !((w[h] >> (8 * i)) & 0xFFu)) w[h] |= 1u << (8 * i);
            }
        }
    store_codes<WHOLE>((uint8_t*)t.m + at, n, mc);
    store_codes<WHOLE>((uint8_t*)t.v + at, n, make_uint2(w[0], w[1]));
    if (lane == 0 && SS1_IN(block, (t.n + kBlock - 1) / kBlock, kSiteAdamScale)) {
        t.m_scale[block] = ms;
        t.v_scale[block] = vs;
    }
}

template <int BITS, bool DITHER>
__device__ __forceinline__ void update_chunk(const Entry& t, uint32_t flags, const Factors& f, F2 none, uint32_t key, int64_t start, int warp,
                                             int lane) {
#pragma unroll 1
    for (int k = warp; k < kChunk / kBlock; k += kWarps) {
        const int64_t block = start / kBlock + k, at = block * kBlock + lane * 8;
        if (block * kBlock >= t.n) break;
        if ((flags & kAligned) && (block + 1) * kBlock <= t.n && SS1_SPAN_IN(at, 8, t.n, kSiteAdamTensor)) {
            update8<BITS, DITHER, true>(t, flags, f, none, key, at, 8, block, lane);
        } else {
            const int64_t left = t.n - at;
            update8<BITS, DITHER, false>(t, flags, f, none, key, left > 0 ? at : 0, left >= 8 ? 8 : (left > 0 ? (int)left : 0), block, lane);
        }
    }
}

template <int N, int BITS>
__global__ void __launch_bounds__(kWarps * 32, 4) adamw_kernel(const __grid_constant__ Table<N> table, const Factors host,
                                                            const float* __restrict__ device, int64_t step,
                                                            const int64_t* __restrict__ device_step, float minus_zero) {
    wait_for_previous();
    const F2 none = F2::both(minus_zero);
    Factors f = host;
    if (device) {
        float* to = reinterpret_cast<float*>(&f);
#pragma unroll
        for (int i = 0; i < kFactors; ++i) to[i] = __ldg(device + i);
    }
    bool dither = false;
    uint32_t key = 0;
    if (BITS == 8) {
        if (device_step) step += __ldg(device_step);
        dither = step > kNearest;
        key = step_key(step);
    }
    // the tensor whose chunks contain this CTA's: the last one that starts at or before it
    int lo = 0, hi = table.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (table.first[mid] <= (int)blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const Entry t = table.t[lo];
    const uint32_t flags = table.flags[lo];
    const int64_t start = (int64_t)((int)blockIdx.x - table.first[lo]) * kChunk;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (BITS == 8 && dither) update_chunk<BITS, BITS == 8>(t, flags, f, none, key, start, warp, lane);
    else update_chunk<BITS, false>(t, flags, f, none, key, start, warp, lane);
}

template <int N>
cudaError_t launch(const ss1_adamw_tensor* tensors, int64_t count, int bits, const Factors& f,
                   const float* device, int64_t step, const int64_t* device_step, cudaStream_t st) {
    static_assert(sizeof(Table<N>) + sizeof(Factors) + 48 <= 32764, "kernel parameters");
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
    // dependent like launch_dependent's, with the table's address instead of copies of it
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)chunks);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    Factors factors = f;
    float minus_zero = -0.0f;
    void* args[] = {&table, &factors, &device, &step, &device_step, &minus_zero};
    return cudaLaunchKernelExC(&cfg, bits == 32 ? reinterpret_cast<const void*>(&adamw_kernel<N, 32>)
                                                : reinterpret_cast<const void*>(&adamw_kernel<N, 8>), args);
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

struct Range {
    uintptr_t lo, hi;
    bool written;
};

// Whether something that the step writes overlaps anything else of it: the CTAs of all tensors run at once. `r`: 7 places a tensor.
bool overlaps(const ss1_adamw_tensor* tensors, int64_t count, int bits, Range* r) {
    Range* end = r;
    auto add = [&end](const void* p, int64_t n, size_t size, bool written) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (p) *end++ = Range{lo, lo + (uintptr_t)n * size, written};
    };
    for (int64_t i = 0; i < count; ++i) {
        const ss1_adamw_tensor& t = tensors[i];
        if (t.numel == 0) continue;
        const size_t state = bits == 32 ? 4 : 1;
        add(t.param, t.numel, dtype_size(t.param_dtype), true);
        if (t.grad != t.param || t.grad_dtype != t.param_dtype) add(t.grad, t.numel, dtype_size(t.grad_dtype), false);
        add(t.master, t.numel, 4, true);
        add(t.exp_avg, t.numel, state, true);
        add(t.exp_avg_sq, t.numel, state, true);
        if (bits == 8) {
            add(t.avg_scale, (t.numel + kBlock - 1) / kBlock, 4, true);
            add(t.sq_scale, (t.numel + kBlock - 1) / kBlock, 4, true);
        }
    }
    std::sort(r, end, [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t any = 0, written = 0;      // ends of what lies before
    for (; r < end; ++r) {
        if (r->lo < written || (r->written && r->lo < any)) return true;
        any = std::max(any, r->hi);
        if (r->written) written = std::max(written, r->hi);
    }
    return false;
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
    return ss1_adamw_step_ex(tensors, count, state_bits, hyper, device_factors, nullptr, stream);
}

extern "C" SS1_API int ss1_adamw_step_ex(const ss1_adamw_tensor* tensors, int64_t count, int state_bits, const ss1_adamw_hyper* hyper,
                                         const float* device_factors, const int64_t* device_step, void* stream) {
    if (count < 0 || (count > 0 && !tensors) || (state_bits != 32 && state_bits != 8)) return SS1_ERR_INVALID_ARG;
    if (!device_factors && !hyper_ok(hyper)) return SS1_ERR_INVALID_ARG;
    if (device_step && !device_factors) return SS1_ERR_INVALID_ARG;
    if (!aligned(device_factors, 4) || !aligned(device_step, 8)) return SS1_ERR_MISALIGNED;
    // rounding by a step number that a replayed graph repeats would hold its moments still
    if (state_bits == 8 && device_factors && !device_step) return SS1_ERR_INVALID_ARG;
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
    Range* const ranges = static_cast<Range*>(malloc((size_t)count * 7 * sizeof(Range) + 1));
    if (!ranges) return SS1_ERR_OUT_OF_MEMORY;
    const bool bad = overlaps(tensors, count, state_bits, ranges);
    free(ranges);
    if (bad) return SS1_ERR_OVERLAP;
    Factors f = {};
    if (!device_factors) f = factors(*hyper);
    const int64_t step = hyper ? hyper->step : 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    for (int64_t at = 0; at < count;) {
        // as many tensors as one launch takes, and no more chunks than its grid can count
        int64_t end = at, chunks = 0;
        for (; end < count && end - at < kLarge; ++end) {
            const int64_t c = (tensors[end].numel + kChunk - 1) / kChunk;
            if (end > at && chunks + c > 0x7FFFFFFF) break;
            chunks += c;
        }
        const cudaError_t e = end - at <= kSmall ? launch<kSmall>(tensors + at, end - at, state_bits, f, device_factors, step, device_step, st)
                                                 : launch<kLarge>(tensors + at, end - at, state_bits, f, device_factors, step, device_step, st);
        if (e != cudaSuccess) { cudaGetLastError(); return SS1_ERR_CUDA; }
        at = end;
    }
    return SS1_OK;
}
