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
    float eps, per_dim;   // 1 / dim
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

// Eight elements of a row as they lie in memory (16 bytes, or 32 of a 32-bit type, by one load).
constexpr int kVec = 8;
template <typename T> struct Raw { uint4 v; };
template <> struct Raw<float> { uint4 v, w; };
__device__ __forceinline__ void load(Raw<float> &r, const float *p) {
    asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.v.x), "=r"(r.v.y), "=r"(r.v.z), "=r"(r.v.w), "=r"(r.w.x), "=r"(r.w.y), "=r"(r.w.z), "=r"(r.w.w)
                 : "l"(p) : "memory");
}
template <typename T> __device__ __forceinline__ void load(Raw<T> &r, const T *p) { r.v = __ldcs((const uint4 *)p); }
__device__ __forceinline__ void clear(Raw<float> &r) { r.v = r.w = make_uint4(0, 0, 0, 0); }
template <typename T> __device__ __forceinline__ void clear(Raw<T> &r) { r.v = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void unpack(const Raw<float> &r, float (&v)[kVec]) {
    const float *p = (const float *)&r;
#pragma unroll
    for (int i = 0; i < kVec; i++) v[i] = p[i];
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16> &r, float (&v)[kVec]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = __bfloat1622float2(((const __nv_bfloat162 *)&r)[i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void unpack(const Raw<__half> &r, float (&v)[kVec]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = __half22float2(((const __half2 *)&r)[i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void store(float *p, const float (&v)[kVec]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
}
template <typename T> __device__ __forceinline__ void store(T *p, const float (&v)[kVec]) { *(uint4 *)p = pack16(v, T()); }
template <typename T>
__device__ __forceinline__ void load_weight(const T *w, float (&out)[kVec]) {
    constexpr int kPart = 16 / sizeof(T) < kVec ? 16 / sizeof(T) : kVec;
#pragma unroll
    for (int i = 0; i < kVec; i += kPart) {
        struct alignas(kPart * sizeof(T)) Part { T v[kPart]; };
        const Part p = *reinterpret_cast<const Part *>(w + i);
#pragma unroll
        for (int j = 0; j < kPart; j++) out[i + j] = to_f32(p.v[j]);
    }
}

// Rows whose parts start where one load can begin.  One CTA per row, kPer groups
// of 8 elements a thread: the row is read once, all loads of a thread before its
// first use, and its 32-bit sums stay in registers between the norm and the
// rounding.  A block of 128 columns is 16 lanes of one warp, so its scale costs
// one short reduction.  HBM is the bound; CTAs are kept small, two groups a
// thread, so that several rows share an SM and one row's reduction runs under
// another's loads (8,192 rows of 4,096 bf16: 40.2 us; four groups 42.3).  With
// quotients rounded to nearest 40.6 us, 5.8 TB/s.
template <typename T, typename W, int kPer>
__global__ void __launch_bounds__(1024) k_head_norm_vec(NormParams P) {
    constexpr int kLanes = kBlock / kVec;
    __shared__ float red[32];
    const uint64_t row = blockIdx.x;
    const uint32_t n = P.dim / kVec;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T *x = (const T *)P.x + row * P.x_stride, *r = (const T *)P.r + row * P.r_stride;
    T *ro = (T *)P.ro + row * P.ro_stride;
    Raw<T> vx[kPer], vr[kPer];   // past the row's end: zeros, which change nothing
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        const uint32_t i = threadIdx.x + j * blockDim.x;
        clear(vx[j]);
        clear(vr[j]);
        if (i < n) {
            load(vx[j], x + i * kVec);
            if (P.r) load(vr[j], r + i * kVec);
        }
    }
    float s[kPer][kVec], sq = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        const uint32_t i = threadIdx.x + j * blockDim.x;
        float a[kVec], b[kVec];
        unpack(vx[j], a);
        unpack(vr[j], b);
#pragma unroll
        for (int c = 0; c < kVec; c++) {
            s[j][c] = P.r ? a[c] + b[c] : a[c];   // x + 0 would lose the sign of -0
            sq = fmaf(s[j][c], s[j][c], sq);
        }
        if (P.ro && i < n) store(ro + i * kVec, s[j]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sq += __shfl_xor_sync(kFull, sq, d);
    if (lane == 0) red[warp] = sq;
    __syncthreads();
    const int warps = blockDim.x / 32;
    sq = lane < warps ? red[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sq += __shfl_xor_sync(kFull, sq, d);
    const float inv = rsqrtf(sq * P.per_dim + P.eps);
    uint8_t *y8 = P.y8 + row * P.y8_stride;
    float *scales = P.scales + row * P.s_row;
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        const uint32_t i = threadIdx.x + j * blockDim.x;
        float w[kVec], amax = 0.0f;
#pragma unroll
        for (int c = 0; c < kVec; c++) w[c] = 0.0f;
        if (i < n) load_weight<W>((const W *)P.w + i * kVec, w);
#pragma unroll
        for (int c = 0; c < kVec; c++) {
            s[j][c] = s[j][c] * inv * w[c];
            amax = max_nan(amax, fabsf(s[j][c]));
        }
        if (i >= n) amax = 0.0f;   // 0 times an infinite 1 / rms is no element of the row
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(kFull, amax, d));
        const float scale = block_scale(amax);
        const Divisor by(scale);
        if (i < n) {
            struct alignas(kVec) Bytes { __nv_fp8x2_storage_t v[kVec / 2]; } b;
#pragma unroll
            for (int c = 0; c < kVec; c += 2)
                b.v[c / 2] = __nv_cvt_float2_to_fp8x2(make_float2(by(s[j][c]), by(s[j][c + 1])), __NV_SATFINITE, __NV_E4M3);
            *reinterpret_cast<Bytes *>(y8 + i * kVec) = b;
            if (lane % kLanes == 0) scales[i / kLanes * P.s_blk] = scale;
        }
    }
}

// Any rows.  One CTA per row; the row's 32-bit sums stay in shared memory
// between the norm and the rounding.  Bound by its loads of one element
// (8,192 x 4,095 bf16 with residual: 98 us, 2.4 TB/s).
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
    const float inv = rsqrtf(block_sum(sq, red) * P.per_dim + P.eps);
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t blocks = (P.dim + kBlock - 1) / kBlock;
    const W *w = (const W *)P.w;
    for (uint32_t b = warp; b < blocks; b += kNormThreads / 32) {
        float y[4];
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t i = b * kBlock + j * 32 + lane;
            y[j] = i < P.dim ? s_row[i] * inv * to_f32(w[i]) : 0.0f;
            amax = max_nan(amax, fabsf(y[j]));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(kFull, amax, d));
        const float scale = block_scale(amax);
        const Divisor by(scale);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t i = b * kBlock + j * 32 + lane;
            if (i < P.dim) P.y8[row * P.y8_stride + i] = to_e4m3(by(y[j]));
        }
        if (lane == 0) P.scales[row * P.s_row + b * P.s_blk] = scale;
    }
}

// One CTA per 128 x 128 block of a weight matrix; each warp takes 16 rows.  Runs
// once per matrix: 65,536 x 4,096 f32 in 223 us (6.0 TB/s), bf16 by loads of 2
// bytes in 743 us (1.1 TB/s).
template <typename T>
__global__ void __launch_bounds__(kNormThreads) k_head_quantize(const T *__restrict__ w, uint64_t stride, uint32_t n_tok,
                                                                uint32_t dim, uint8_t *__restrict__ w8, uint64_t w8_stride,
                                                                float *__restrict__ ws, uint64_t ws_stride) {
    __shared__ float red[kNormThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = kNormThreads / 32, kRows = kBlock / kWarps;
    const uint32_t col0 = blockIdx.y * kBlock;
    const uint64_t row0 = (uint64_t)blockIdx.x * kBlock;
    float v[kRows][4], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const uint64_t row = row0 + warp + i * kWarps;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t col = col0 + j * 32 + lane;
            v[i][j] = row < n_tok && col < dim ? to_f32(w[row * stride + col]) : 0.0f;
            amax = max_nan(amax, fabsf(v[i][j]));
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(kFull, amax, d));
    if (lane == 0) red[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; i++) amax = max_nan(amax, red[i]);
    const float scale = block_scale(amax);
    const Divisor by(scale);
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const uint64_t row = row0 + warp + i * kWarps;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t col = col0 + j * 32 + lane;
            if (row < n_tok && col < dim) w8[row * w8_stride + col] = to_e4m3(by(v[i][j]));
        }
    }
    if (threadIdx.x == 0) ws[blockIdx.x * ws_stride + blockIdx.y] = scale;
}

// Whether every row of a matrix starts on `bytes`.
bool rows_start_on(const void *p, uint64_t stride, size_t element, uint32_t n_rows, size_t bytes) {
    return (uintptr_t)p % bytes == 0 && (n_rows == 1 || stride * element % bytes == 0);
}

template <typename T>
int launch_norm(bpe_ctx *ctx, const NormParams &P, uint32_t n_rows, int weight_type) {
    constexpr size_t kBytes = kVec * sizeof(T);
    if (P.dim % kVec == 0 && (uintptr_t)P.w % 16 == 0 && rows_start_on(P.x, P.x_stride, sizeof(T), n_rows, kBytes) &&
        (!P.r || rows_start_on(P.r, P.r_stride, sizeof(T), n_rows, kBytes)) &&
        (!P.ro || rows_start_on(P.ro, P.ro_stride, sizeof(T), n_rows, kBytes)) && rows_start_on(P.y8, P.y8_stride, 1, n_rows, kVec)) {
        const uint32_t n = P.dim / kVec, per = n > 2048 ? 4 : 2;
        uint32_t threads = 32;
        while (threads * per < n) threads *= 2;
        auto k2 = weight_type == BPE_F32 ? k_head_norm_vec<T, float, 2>
                  : weight_type == BPE_BF16 ? k_head_norm_vec<T, __nv_bfloat16, 2> : k_head_norm_vec<T, __half, 2>;
        auto k4 = weight_type == BPE_F32 ? k_head_norm_vec<T, float, 4>
                  : weight_type == BPE_BF16 ? k_head_norm_vec<T, __nv_bfloat16, 4> : k_head_norm_vec<T, __half, 4>;
        (per == 4 ? k4 : k2)<<<n_rows, threads, 0, ctx->stream>>>(P);
        BPE_CUDA(ctx, cudaGetLastError(), "head_norm launch");
        return BPE_OK;
    }
    auto k = weight_type == BPE_F32 ? k_head_norm<T, float>
             : weight_type == BPE_BF16 ? k_head_norm<T, __nv_bfloat16> : k_head_norm<T, __half>;
    const size_t smem = (size_t)P.dim * sizeof(float);
    // Beyond what any kernel has, 48 KB together with its static arrays.  The limit is the device's, for all contexts and
    // threads: always raised to the largest row's, never lowered.
    static std::atomic<uint64_t> devices[3];   // of each weight type's kernel
    if (smem > 32 * 1024)
        BPE_CUDA(ctx, allow_shared(k, ctx->device, BPE_HEAD_MAX_DIM * sizeof(float), devices[weight_type]), "head_norm");
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
                 residual_out_stride, y8_stride, scale_row_stride, scale_block_stride, dim, eps, 1.0f / (float)dim};
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
