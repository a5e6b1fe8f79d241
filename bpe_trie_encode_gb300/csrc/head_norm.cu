// head_norm.cu -- residual addition, root-mean-square norm and 8-bit output
// with a scale per 128 columns; and the 8-bit form of a weight matrix.
#include "head.cuh"

#include "device.cuh"
#include "internal.h"

namespace bpe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kBlock = (int)BPE_HEAD_BLOCK;

struct NormParams {
    const void *x, *w, *r;
    void *ro;
    uint8_t *y8;
    float *scales;
    uint64_t x_stride, r_stride, ro_stride, y8_stride, s_row, s_blk;
    uint32_t dim;
    float eps;
};

__device__ __forceinline__ float block_sum(float v, float *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; i++) t += red[i];
    return t;
}

// One CTA per row; the row's 32-bit sums stay in shared memory between the
// norm and the rounding.
template <typename T, typename W>
__global__ void __launch_bounds__(kNormThreads) k_head_norm(NormParams P) {
    extern __shared__ float s_row[];
    __shared__ float red[kNormThreads / 32];
    const uint64_t row = blockIdx.x;
    const T *x = (const T *)P.x + row * P.x_stride;
    const T *r = P.r ? (const T *)P.r + row * P.r_stride : nullptr;
    T *ro = P.ro ? (T *)P.ro + row * P.ro_stride : nullptr;
    float sq = 0.0f;
    for (uint32_t i = threadIdx.x; i < P.dim; i += kNormThreads) {
        float v = to_f32(x[i]);
        if (r) v += to_f32(r[i]);
        if (ro) ro[i] = from_f32<T>(v);
        s_row[i] = v;
        sq = fmaf(v, v, sq);
    }
    const float inv = rsqrtf(block_sum(sq, red) / (float)P.dim + P.eps);
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t blocks = (P.dim + kBlock - 1) / kBlock;
    const W *w = (const W *)P.w;
    for (uint32_t b = warp; b < blocks; b += kNormThreads / 32) {
        float y[4];
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t i = b * kBlock + j * 32 + lane;
            y[j] = i < P.dim ? s_row[i] * inv * to_f32(w[i]) : 0.0f;
            amax = max(amax, abs_bits(y[j]));
        }
        amax = __reduce_max_sync(kFull, amax);
        const float scale = block_scale(amax), back = 1.0f / scale;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t i = b * kBlock + j * 32 + lane;
            if (i < P.dim) P.y8[row * P.y8_stride + i] = to_e4m3(y[j] * back);
        }
        if (lane == 0) P.scales[row * P.s_row + b * P.s_blk] = scale;
    }
}

// One CTA per 128 x 128 block of a weight matrix; each warp takes 16 rows.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) k_head_quantize(const T *__restrict__ w, uint64_t stride, uint32_t n_tok,
                                                                uint32_t dim, uint8_t *__restrict__ w8, uint64_t w8_stride,
                                                                float *__restrict__ ws, uint64_t ws_stride) {
    __shared__ uint32_t red[kNormThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = kNormThreads / 32, kRows = kBlock / kWarps;
    const uint32_t col0 = blockIdx.y * kBlock;
    const uint64_t row0 = (uint64_t)blockIdx.x * kBlock;
    float v[kRows][4];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const uint64_t row = row0 + warp + i * kWarps;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t col = col0 + j * 32 + lane;
            v[i][j] = row < n_tok && col < dim ? to_f32(w[row * stride + col]) : 0.0f;
            amax = max(amax, abs_bits(v[i][j]));
        }
    }
    amax = __reduce_max_sync(kFull, amax);
    if (lane == 0) red[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; i++) amax = max(amax, red[i]);
    const float scale = block_scale(amax), back = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const uint64_t row = row0 + warp + i * kWarps;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t col = col0 + j * 32 + lane;
            if (row < n_tok && col < dim) w8[row * w8_stride + col] = to_e4m3(v[i][j] * back);
        }
    }
    if (threadIdx.x == 0) ws[blockIdx.x * ws_stride + blockIdx.y] = scale;
}

template <typename T>
int launch_norm(bpe_ctx *ctx, const NormParams &P, uint32_t n_rows, int weight_type) {
    auto k = weight_type == BPE_F32 ? k_head_norm<T, float>
             : weight_type == BPE_BF16 ? k_head_norm<T, __nv_bfloat16> : k_head_norm<T, __half>;
    const size_t smem = (size_t)P.dim * sizeof(float);
    if (smem > 48 * 1024)
        BPE_CUDA(ctx, cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem), "head_norm");
    k<<<n_rows, kNormThreads, smem, ctx->stream>>>(P);
    BPE_CUDA(ctx, cudaGetLastError(), "head_norm launch");
    return BPE_OK;
}

}  // namespace
}  // namespace bpe

using namespace bpe;

extern "C" int head_norm(bpe_ctx *ctx, const void *d_x, uint64_t x_stride, int type, const void *d_weight, int weight_type,
                         const void *d_residual, uint64_t residual_stride, uint32_t n_rows, uint32_t dim, float eps,
                         void *d_residual_out, uint64_t residual_out_stride, uint8_t *d_y8, uint64_t y8_stride,
                         float *d_scales, uint64_t scale_row_stride, uint64_t scale_block_stride) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    if (!head_type_ok(type) || !head_type_ok(weight_type))
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_norm: unknown element type");
    if (dim == 0 || dim > BPE_HEAD_MAX_DIM)
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_norm: dim %u outside 1..%u", dim, BPE_HEAD_MAX_DIM);
    if (!(eps >= 0.0f)) return fail(ctx, BPE_ERR_INVALID_ARG, "head_norm: eps is negative or NaN");
    if (n_rows == 0) return BPE_OK;
    if (n_rows > 0x7FFFFFFFu) return fail(ctx, BPE_ERR_INVALID_ARG, "head_norm: %u rows", n_rows);
    if (!d_x || !d_weight || !d_y8 || !d_scales) return fail(ctx, BPE_ERR_INVALID_ARG, "head_norm: null pointer");
    if (n_rows > 1 && (x_stride < dim || y8_stride < dim || (d_residual && residual_stride < dim) ||
                       (d_residual_out && residual_out_stride < dim)))
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_norm: a row stride is below dim %u", dim);
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    NormParams P{d_x, d_weight, d_residual, d_residual_out, d_y8, d_scales, x_stride, residual_stride,
                 residual_out_stride, y8_stride, scale_row_stride, scale_block_stride, dim, eps};
    if (type == BPE_F32) return launch_norm<float>(ctx, P, n_rows, weight_type);
    if (type == BPE_BF16) return launch_norm<__nv_bfloat16>(ctx, P, n_rows, weight_type);
    return launch_norm<__half>(ctx, P, n_rows, weight_type);
}

extern "C" int head_quantize(bpe_ctx *ctx, const void *d_w, uint64_t w_stride, int type, uint32_t n_tok, uint32_t dim,
                             uint8_t *d_w8, uint64_t w8_stride, float *d_ws, uint64_t ws_stride) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    if (!head_type_ok(type)) return fail(ctx, BPE_ERR_INVALID_ARG, "head_quantize: unknown element type");
    if (dim == 0 || dim > BPE_HEAD_MAX_DIM || n_tok == 0 || n_tok > BPE_HEAD_MAX_TOKENS)
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_quantize: %u tokens of %u columns", n_tok, dim);
    const uint32_t blocks = (dim + kBlock - 1) / kBlock;
    if (!d_w || !d_w8 || !d_ws) return fail(ctx, BPE_ERR_INVALID_ARG, "head_quantize: null pointer");
    if ((n_tok > 1 && (w_stride < dim || w8_stride < dim)) || (n_tok > BPE_HEAD_BLOCK && ws_stride < blocks))
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_quantize: a row stride is too small");
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    const dim3 grid((n_tok + kBlock - 1) / kBlock, blocks);
    cudaStream_t s = ctx->stream;
    if (type == BPE_F32)
        k_head_quantize<float><<<grid, kNormThreads, 0, s>>>((const float *)d_w, w_stride, n_tok, dim, d_w8, w8_stride, d_ws, ws_stride);
    else if (type == BPE_BF16)
        k_head_quantize<__nv_bfloat16><<<grid, kNormThreads, 0, s>>>((const __nv_bfloat16 *)d_w, w_stride, n_tok, dim, d_w8, w8_stride, d_ws, ws_stride);
    else
        k_head_quantize<__half><<<grid, kNormThreads, 0, s>>>((const __half *)d_w, w_stride, n_tok, dim, d_w8, w8_stride, d_ws, ws_stride);
    BPE_CUDA(ctx, cudaGetLastError(), "head_quantize launch");
    return BPE_OK;
}
