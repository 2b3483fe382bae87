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
// nearest even.
struct KvInt8 {
    __device__ static constexpr float top() { return 127.0f; }
    __device__ __forceinline__ static float value(uint8_t c) {
        return static_cast<float>(static_cast<int8_t>(c));
    }
    __device__ __forceinline__ static uint8_t code(float y) {  // NaN -> 0
        y = y == y ? fminf(fmaxf(rintf(y), -127.0f), 127.0f) : 0.0f;
        return static_cast<uint8_t>(static_cast<int8_t>(static_cast<int>(y)));
    }
};
struct KvE4m3 {
    __device__ static constexpr float top() { return 448.0f; }
    __device__ __forceinline__ static float value(uint8_t c) {
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
    }
    __device__ __forceinline__ static uint8_t code(float y) {
        return y == y ? __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3) : 0;
    }
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// Sequence and index within it of slot x, where sequence i owns slots
// cu[i] / B + 2 i onwards: at least as many as the pages of B tokens that its
// cu[i+1] - cu[i] consecutive positions can touch.
__device__ __forceinline__ int seq_of_slot(const int32_t* __restrict__ cu, int n, int B, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] / B + 2 * mid <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
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
