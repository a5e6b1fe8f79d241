// head_logits.cu -- 8-bit matrix product with a scale per block of 128.
#include "head.cuh"

#include "device.cuh"
#include "internal.h"

namespace bpe {
namespace {

constexpr int kBlock = (int)BPE_HEAD_BLOCK;
constexpr int kTile = 64, kDepth = 32;   // output tile, columns staged at a time

struct LogitsParams {
    const uint8_t *x8, *w8;
    const float *xs, *ws;
    void *out;
    uint64_t x_stride, xs_row, xs_blk, w_stride, ws_row, ws_blk, out_stride;
    uint32_t n_rows, n_tok, dim;
};

// One CTA per 64 x 64 tile of the output, 4 x 4 per thread.
template <typename O>
__global__ void __launch_bounds__(256) k_head_logits(LogitsParams P) {
    __shared__ float sx[kDepth][kTile + 1], sw[kDepth][kTile + 1];
    const uint32_t row0 = blockIdx.y * kTile, tok0 = blockIdx.x * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {}, part[4][4] = {};
    for (uint32_t k0 = 0; k0 < P.dim; k0 += kDepth) {
        for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
            const uint32_t r = i / kDepth, c = i % kDepth, k = k0 + c;
            __nv_fp8_e4m3 a, b;
            a.__x = row0 + r < P.n_rows && k < P.dim ? P.x8[(row0 + r) * P.x_stride + k] : 0;
            b.__x = tok0 + r < P.n_tok && k < P.dim ? P.w8[(uint64_t)(tok0 + r) * P.w_stride + k] : 0;
            sx[c][r] = (float)a;
            sw[c][r] = (float)b;
        }
        __syncthreads();
#pragma unroll 8
        for (int c = 0; c < kDepth; c++) {
            float a[4], b[4];
#pragma unroll
            for (int j = 0; j < 4; j++) a[j] = sx[c][ty + 16 * j], b[j] = sw[c][tx + 16 * j];
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) part[i][j] = fmaf(a[i], b[j], part[i][j]);
        }
        __syncthreads();
        if ((k0 + kDepth) % kBlock == 0 || k0 + kDepth >= P.dim) {
            const uint32_t blk = k0 / kBlock;
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint32_t r = row0 + ty + 16 * i, t = tok0 + tx + 16 * j;
                    const float s = r < P.n_rows && t < P.n_tok
                        ? P.xs[r * P.xs_row + blk * P.xs_blk] * P.ws[t / kBlock * P.ws_row + blk * P.ws_blk] : 0.0f;
                    acc[i][j] = fmaf(part[i][j], s, acc[i][j]);
                    part[i][j] = 0.0f;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t r = row0 + ty + 16 * i, t = tok0 + tx + 16 * j;
            if (r < P.n_rows && t < P.n_tok) ((O *)P.out)[r * P.out_stride + t] = from_f32<O>(acc[i][j]);
        }
}

}  // namespace
}  // namespace bpe

using namespace bpe;

extern "C" int head_logits(bpe_ctx *ctx, const uint8_t *d_x8, uint64_t x8_stride, const float *d_xs, uint64_t xs_row_stride,
                           uint64_t xs_block_stride, const uint8_t *d_w8, uint64_t w8_stride, const float *d_ws,
                           uint64_t ws_row_stride, uint64_t ws_block_stride, uint32_t n_rows, uint32_t n_tok, uint32_t dim,
                           void *d_out, uint64_t out_stride, int out_type) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    if (!head_type_ok(out_type)) return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: unknown output type");
    if (dim == 0 || dim > BPE_HEAD_MAX_DIM || n_tok == 0 || n_tok > BPE_HEAD_MAX_TOKENS)
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: %u tokens of %u columns", n_tok, dim);
    if (n_rows == 0) return BPE_OK;
    if (n_rows > (1u << 22)) return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: %u rows", n_rows);
    if (!d_x8 || !d_xs || !d_w8 || !d_ws || !d_out) return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: null pointer");
    if ((n_rows > 1 && (x8_stride < dim || out_stride < n_tok)) || (n_tok > 1 && w8_stride < dim))
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: a row stride is below its row's length");
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    LogitsParams P{d_x8, d_w8, d_xs, d_ws, d_out, x8_stride, xs_row_stride, xs_block_stride, w8_stride,
                   ws_row_stride, ws_block_stride, out_stride, n_rows, n_tok, dim};
    const dim3 grid((n_tok + kTile - 1) / kTile, (n_rows + kTile - 1) / kTile);
    if (grid.y > 65535) return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: %u rows", n_rows);
    if (out_type == BPE_F32)
        k_head_logits<float><<<grid, 256, 0, ctx->stream>>>(P);
    else if (out_type == BPE_BF16)
        k_head_logits<__nv_bfloat16><<<grid, 256, 0, ctx->stream>>>(P);
    else
        k_head_logits<__half><<<grid, 256, 0, ctx->stream>>>(P);
    BPE_CUDA(ctx, cudaGetLastError(), "head_logits launch");
    return BPE_OK;
}
