// head.cuh -- element types and small helpers shared by the output head's
// kernels (head_norm.cu, head_logits.cu, head_sample.cu).
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

// |v| as an ordered whole number: the order of magnitudes, with infinity above
// every finite value and NaN above infinity, so that a maximum keeps them.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Scale of a block whose largest magnitude has the bits `amax`.
__device__ __forceinline__ float block_scale(uint32_t amax) {
    const float s = __uint_as_float(amax) / kE4m3Max;
    return s < kMinScale ? kMinScale : s;   // NaN stays
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
