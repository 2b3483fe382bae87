// Device helpers of the paged 8-bit cache: codes to values and back.
#pragma once

#include <atomic>

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_common.cuh"
#include "gdn_kv.h"

namespace gdn {

// Cache codes.  top: the largest code value; a block's scale is its largest
// |value| times 1 / top (one fp32 product), a code is value / scale rounded to
// nearest even, saturating, NaN as 0.
struct KvInt8 {
    __device__ static constexpr float top() { return 127.0f; }
    __device__ __forceinline__ static float value(uint8_t c) {
        return static_cast<float>(static_cast<int8_t>(c));
    }
    __device__ __forceinline__ static uint32_t code4(const float* y) {
        int v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = max(min(__float2int_rn(y[i]), 127), -127);  // NaN converts to 0
        return __byte_perm(__byte_perm(v[0], v[1], 0x0040), __byte_perm(v[2], v[3], 0x0040), 0x5410);
    }
};
struct KvE4m3 {
    __device__ static constexpr float top() { return 448.0f; }
    __device__ __forceinline__ static float value(uint8_t c) {
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
    }
    __device__ __forceinline__ static uint32_t code4(const float* y) {
        float z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = y[i] == y[i] ? y[i] : 0.0f;
        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(z[0], z[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(z[2], z[3]), __NV_SATFINITE, __NV_E4M3);
        return a | b << 16;
    }
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Values of a block whose scale is 0 add nothing to the output, but their weights
// count in the softmax's sum, as 2^(score - reference).  They move the reference
// only as if their scale were 2^-kZeroLog: values of a larger one lift it as soon
// as they come, and keep their weights' bits.  (A weight of the sum is then at
// most 2^(15 + kZeroLog), and 2^21 of them are an fp32 number.)
constexpr float kZeroLog = 90.0f;
// Scales below 2^-kZeroLog count as 0: a reciprocal of up to 2^kZeroLog leaves a
// sum of 2^21 weights an fp32 number (that of a subnormal scale is infinite).  What
// is lost is below 2^-81 in magnitude.
__device__ __forceinline__ bool zero_scale(float s) { return s >= 0.0f && s < 8.07793567e-28f; }

// l 2^x, x <= 0, given f = 2^x: the sums above span more than fp32's normal
// numbers reach to one side, so that f may be flushed to 0 where the product is not.
__device__ __forceinline__ float times_pow2(float l, float x, float f) {
    return x >= -100.0f ? l * f : l * 7.88860905e-31f * exp2_ftz(x + 100.0f);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Four codes of a word to f16: codes (0, 1) and (2, 3).
template <typename F> __device__ __forceinline__ void widen_f16(uint32_t w, uint32_t& a, uint32_t& b);
template <> __device__ __forceinline__ void widen_f16<KvInt8>(uint32_t w, uint32_t& a, uint32_t& b) {
    // bytes u = code + 128 under the exponent of 1024 are the f16 1024 + u; less 1152 it is the code
    w ^= 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    uint32_t x = __byte_perm(w, 0x64646464u, 0x4140), y = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 hx = __hsub2(*reinterpret_cast<__half2*>(&x), off), hy = __hsub2(*reinterpret_cast<__half2*>(&y), off);
    a = *reinterpret_cast<const uint32_t*>(&hx);
    b = *reinterpret_cast<const uint32_t*>(&hy);
}
template <> __device__ __forceinline__ void widen_f16<KvE4m3>(uint32_t w, uint32_t& a, uint32_t& b) {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
}

// The largest i in 0 .. n - 1 with key(i) <= x (key does not decrease, key(0) <=
// x), by the whole warp: one load for up to 32 sequences, two for up to 1024.
template <typename K> __device__ __forceinline__ int warp_search(int n, int x, K&& key) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) / 32, at = lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < n && key(lo + at) <= x);
        const int k = 31 - __clz(below);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}
// The sequence of packed token t, by a warp.
__device__ __forceinline__ int warp_seq_of_token(const int32_t* __restrict__ cu, int n, int t) {
    return warp_search(n, t, [&](int i) { return cu[i]; });
}
// The sequence of slot x, where sequence i owns slots cu[i] / B + 2 i onwards: at
// least as many as the pages of B tokens that its cu[i+1] - cu[i] consecutive
// positions can touch.
__device__ __forceinline__ int warp_seq_of_slot(const int32_t* __restrict__ cu, int n, int B, int x) {
    return warp_search(n, x, [&](int i) { return cu[i] / B + 2 * i; });
}

// Lets `kernel` use `bytes` of dynamic shared memory, once per device (ready:
// one bit per device; devices past 63 ask every time).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<unsigned long long>& ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Instantiates a launcher fn<activation type, code format, head dim>(a, stream)
// for the names bf16, e4m3 and head_dim in scope.
#define GDN_KV_PICK_D(fn, T, F)                                    \
    (head_dim == 64 ? fn<T, F, 64>(a, stream)                      \
                    : head_dim == 128 ? fn<T, F, 128>(a, stream) : fn<T, F, 256>(a, stream))
#define GDN_KV_PICK(fn)                                                                        \
    (bf16 ? (e4m3 ? GDN_KV_PICK_D(fn, __nv_bfloat16, KvE4m3) : GDN_KV_PICK_D(fn, __nv_bfloat16, KvInt8)) \
          : (e4m3 ? GDN_KV_PICK_D(fn, float, KvE4m3) : GDN_KV_PICK_D(fn, float, KvInt8)))

}  // namespace gdn
