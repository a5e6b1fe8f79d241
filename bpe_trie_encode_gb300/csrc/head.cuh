// head.cuh -- element types and small helpers shared by the output head's
// kernels (head_norm.cu, head_logits.cu, head_sample.cu, head_score.cu,
// head_distill.cuh).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <cstdint>

#include "bpetrie.h"

namespace bpe {

constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126, the smallest normal number

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// The larger of two, a NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Scale of a block whose largest magnitude is `amax`: a product with the 32-bit number next to 1 / 448; NaN stays.
__device__ __forceinline__ float block_scale(float amax) {
    return max_nan(amax * (1.0f / kE4m3Max), kMinScale);
}

// Quotients by a block's scale, rounded to nearest.  With r near 1 / scale and e = 1 - scale r, which one fused step gives
// without rounding, 1 / scale = r + r e + ... (the geometric series; the next term is 2^-46 of it), so that v / scale is
// v r + v (r e), rounded once: of 10^10 random pairs some 50 were off in the last bit below scales of 2^73, and no 8-bit
// value was.  A product with a 32-bit reciprocal alone is off there for one value in three, and where that bit lies on a
// tie of the 8-bit numbers the value is a step off.  The division function costs registers here, and with them CTAs on an
// SM (8,192 x 4,096 f32: 36.6 us with it once a block, 34.2 so).  By an infinite scale: NaN.
struct Divisor {
    float r, re;
    __device__ __forceinline__ explicit Divisor(float scale) {
        r = __fdividef(1.0f, scale);
        re = r * fmaf(-scale, r, 1.0f);
    }
    __device__ __forceinline__ float operator()(float v) const { return fmaf(v, r, v * re); }
};

// 16 bytes of a type from 32-bit values.
__device__ __forceinline__ uint4 pack16(const float *v, float) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack16(const float *v, __nv_bfloat16) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    __nv_bfloat162 c = __floats2bfloat162_rn(v[4], v[5]), d = __floats2bfloat162_rn(v[6], v[7]);
    return make_uint4(*(uint32_t *)&a, *(uint32_t *)&b, *(uint32_t *)&c, *(uint32_t *)&d);
}
__device__ __forceinline__ uint4 pack16(const float *v, __half) {
    __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
    __half2 c = __floats2half2_rn(v[4], v[5]), d = __floats2half2_rn(v[6], v[7]);
    return make_uint4(*(uint32_t *)&a, *(uint32_t *)&b, *(uint32_t *)&c, *(uint32_t *)&d);
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
    return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

// Lets a kernel have `bytes` of shared memory on this device; asked of the runtime once per device.
template <typename K>
inline cudaError_t allow_shared(K kernel, int device, size_t bytes, std::atomic<uint64_t> &devices) {
    const uint64_t bit = 1ull << (device & 63);
    if (device < 64 && (devices.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && device < 64) devices.fetch_or(bit, std::memory_order_release);
    return e;
}

inline bool head_type_ok(int t) { return t == BPE_F32 || t == BPE_BF16 || t == BPE_F16; }
inline size_t head_type_size(int t) { return t == BPE_F32 ? 4 : 2; }

}  // namespace bpe
