// Shared by the operators around a projection (layer norm, low-rank adapters, AdamW): element
// conversions, 8-element vector loads and stores, warp sums, pointer checks.
#pragma once

#include "ss1_internal.cuh"

#include <cuda_bf16.h>

namespace ss1 {
namespace op {

// Checked build: access sites of these operators (their numbers follow the layer's sites).
enum Site : int {
    kSiteNormX = 32, kSiteNormW, kSiteNormY, kSiteNormPart,
    kSitePlan, kSiteAdaX, kSiteAdaA, kSiteAdaB, kSiteAdaY, kSiteAdaH, kSiteAdaG, kSiteAdaPart,
    kSiteAdamTensor, kSiteAdamScale,
};

template <typename T>
__device__ __forceinline__ float to_f(T v) { return (float)v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v) { return (T)v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Two floats in one 64-bit register pair: sm_100's packed float32 operations do both at once, each
// rounded as the single one is. The assembler joins a product and a sum into one multiply-add, .rn or not.
struct F2 {
    unsigned long long v;
    __device__ __forceinline__ static F2 of(float lo, float hi) {
        F2 r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
        return r;
    }
    __device__ __forceinline__ static F2 both(float x) { return of(x, x); }
    __device__ __forceinline__ float lo() const { return __uint_as_float((uint32_t)v); }
    __device__ __forceinline__ float hi() const { return __uint_as_float((uint32_t)(v >> 32)); }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Eight consecutive elements, 16-byte aligned, as they lie in memory (bf16: one 16-byte word,
// float: two).
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void load_once(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // a bf16 is the upper half of the float of the same value
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void get(F2 (&f)[4]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = F2::of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ __forceinline__ void set(const F2 (&f)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[i].lo(), f[i].hi());
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void load_once(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p + 4));
    }
    __device__ __forceinline__ void store(float* p) const {
        *reinterpret_cast<float4*>(p) = a;
        *reinterpret_cast<float4*>(p + 4) = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void get(F2 (&f)[4]) const {
        f[0] = F2::of(a.x, a.y); f[1] = F2::of(a.z, a.w); f[2] = F2::of(b.x, b.y); f[3] = F2::of(b.z, b.w);
    }
    __device__ __forceinline__ void set(const F2 (&f)[4]) {
        a = make_float4(f[0].lo(), f[0].hi(), f[1].lo(), f[1].hi());
        b = make_float4(f[2].lo(), f[2].hi(), f[3].lo(), f[3].hi());
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
};

inline bool dtype_ok(int dtype) { return dtype == SS1_DTYPE_BF16 || dtype == SS1_DTYPE_FP32; }
inline size_t dtype_size(int dtype) { return dtype == SS1_DTYPE_BF16 ? 2 : 4; }
inline bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Launches `kernel` so that it may start while the previous kernel on the stream drains
// (programmatic dependent launch). Rules that every kernel launched like this keeps: all its CTAs execute
// griddepcontrol.wait before they end, so that what it has waited for is over for whoever waits for it; and
// before the wait it touches nothing that an earlier kernel may still write. A kernel lets its
// successor start only after its own wait, except where its successor waits first thing; and only where the
// successor has something to do before its wait, because CTAs that merely wait settle unevenly on the
// SMs (layer norm forward 4096 x 4096: 17.4 us with, 15.4 without).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace op
}  // namespace ss1
