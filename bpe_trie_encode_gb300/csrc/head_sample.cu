// head_sample.cu -- temperature, top-k, top-p, min-p and the draw of one id
// per row from a given random number.
#include "head.cuh"

#include "device.cuh"
#include "internal.h"

namespace bpe {
namespace {

constexpr int kSampThreads = 512;
constexpr float kOne = 1099511627776.0f;   // 2^40

typedef unsigned long long u64;

struct SampleParams {
    const void *logits;
    uint64_t stride;
    uint32_t n_tok;
    const float *u;
    head_filters f;
    int32_t *ids;
    float *logprob;
};

// Logits as whole numbers of the same order (a NaN as -infinity, -0 as 0).
constexpr uint32_t kKeyNegInf = 0x007FFFFFu, kKeyPosInf = 0xFF800000u;
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
    return v != v ? kKeyNegInf : k;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float z_of(float v, float top, float inv_t) { return v == top ? 0.0f : (v - top) * inv_t; }
__device__ __forceinline__ u64 weight_of(float v, float top, float inv_t) {
    return v > -INFINITY ? (u64)(expf(z_of(v, top, inv_t)) * kOne) : 0;   // 0 for -infinity and NaN
}

__device__ __forceinline__ u64 sum_all(u64 v, u64 *red) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    u64 t = 0;
    for (int i = 0; i < kSampThreads / 32; i++) t += red[i];
    return t;
}

// One CTA per row.  The kept tokens are those with a key above `cut`, and the
// first `ties` with the key `cut`; the cut is found bit by bit.
template <typename T>
__global__ void __launch_bounds__(kSampThreads) k_head_sample(SampleParams P) {
    __shared__ u64 red[kSampThreads / 32];
    __shared__ u64 seg_mass[kSampThreads / 32];
    __shared__ uint32_t seg_ties[kSampThreads / 32];
    const uint64_t row = blockIdx.x;
    const T *l = (const T *)P.logits + row * P.stride;
    const uint32_t n = P.n_tok;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    uint32_t kmax = kKeyNegInf;
    for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) kmax = max(kmax, key_of(to_f32(l[i])));
    kmax = __reduce_max_sync(kFull, kmax);
    if (lane == 0) seg_ties[warp] = kmax;
    __syncthreads();
    for (int i = 0; i < kSampThreads / 32; i++) kmax = max(kmax, seg_ties[i]);
    __syncthreads();
    if (kmax == kKeyNegInf) {
        if (threadIdx.x == 0) {
            P.ids[row] = -1;
            if (P.logprob) P.logprob[row] = __uint_as_float(0xFF800000u);
        }
        return;
    }
    const float top = key_value(kmax);
    const float temp = P.f.d_temperature ? P.f.d_temperature[row] : P.f.temperature;
    const int32_t k = P.f.d_top_k ? P.f.d_top_k[row] : P.f.top_k;
    const float p = P.f.d_top_p ? P.f.d_top_p[row] : P.f.top_p;
    const float q = P.f.d_min_p ? P.f.d_min_p[row] : P.f.min_p;
    const bool greedy = !(temp >= kMinScale);
    const float inv_t = greedy ? 1.0f : 1.0f / temp;

    uint32_t cut = 0, ties = 0;          // keep all
    const u64 least = q > 0.0f ? (u64)(fminf(q, 1.0f) * kOne) : 0;
    if (greedy) {
        cut = kmax;
        ties = 1;
    } else {
        if (k >= 1 && (uint32_t)k < n) {
            for (int bit = 31; bit >= 0; bit--) {
                const uint32_t c = cut | 1u << bit;
                u64 cnt = 0;
                for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) cnt += key_of(to_f32(l[i])) >= c;
                if (sum_all(cnt, red) >= (u64)k) cut = c;
            }
            u64 above = 0;
            for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) above += key_of(to_f32(l[i])) > cut;
            ties = (uint32_t)((u64)k - sum_all(above, red));
        }
        if (p < 1.0f) {
            u64 mass = 0;
            for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) {
                const float v = to_f32(l[i]);
                if (key_of(v) > cut) mass += weight_of(v, top, inv_t);
            }
            mass = sum_all(mass, red) + (ties ? ties * weight_of(key_value(cut), top, inv_t) : 0);
            const double e = (double)p * (double)mass;
            u64 edge = e > 1.0 ? (u64)e : 1;
            uint32_t c2 = 0;
            for (int bit = 31; bit >= 0; bit--) {
                const uint32_t c = c2 | 1u << bit;
                u64 m = 0;
                for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) {
                    const float v = to_f32(l[i]);
                    if (key_of(v) >= c) m += weight_of(v, top, inv_t);
                }
                if (sum_all(m, red) >= edge) c2 = c;
            }
            u64 above = 0;
            for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) {
                const float v = to_f32(l[i]);
                if (key_of(v) > c2) above += weight_of(v, top, inv_t);
            }
            above = sum_all(above, red);
            const u64 w = weight_of(key_value(c2), top, inv_t);
            const uint32_t t2 = (uint32_t)((edge - above + w - 1) / w);
            if (c2 > cut) cut = c2, ties = t2;
            else if (c2 == cut) ties = min(ties, t2);
        }
    }

    // each warp takes a contiguous segment; mass above the cut and ties in it
    const uint32_t seg = ((n + kSampThreads / 32 - 1) / (kSampThreads / 32) + 31) & ~31u;
    const uint32_t s0 = min(n, warp * seg), s1 = min(n, s0 + seg);
    u64 mass = 0;
    uint32_t eq = 0;
    for (uint32_t i = s0 + lane; i < s1; i += 32) {
        const float v = to_f32(l[i]);
        const uint32_t key = key_of(v);
        const u64 w = key >= cut ? weight_of(v, top, inv_t) : 0;
        if (key > cut && w >= least) mass += w;
        eq += key == cut;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mass += __shfl_xor_sync(kFull, mass, d);
    eq = __reduce_add_sync(kFull, eq);
    if (lane == 0) seg_mass[warp] = mass, seg_ties[warp] = eq;
    __syncthreads();
    u64 wc = ties ? weight_of(key_value(cut), top, inv_t) : 0;
    if (wc < least) wc = 0;
    u64 total = 0;
    uint32_t seen = 0;
    for (int i = 0; i < kSampThreads / 32; i++) total += seg_mass[i], seen += seg_ties[i];
    total += min(seen, ties) * wc;
    const float u = P.u[row];
    const double at = (double)u * (double)total;
    u64 t = at > 0.0 ? (u64)at : 0;
    if (t > total - 1) t = total - 1;
    // the warp whose segment holds it
    u64 before = 0;
    uint32_t eq_before = 0;
    for (int i = 0; i < warp; i++) before += seg_mass[i], eq_before += seg_ties[i];
    const u64 lo = before + min(eq_before, ties) * wc;
    const u64 hi = before + mass + min(eq_before + eq, ties) * wc;
    if (t < lo || t >= hi) return;
    for (uint32_t i0 = s0; i0 < s1; i0 += 32) {
        const uint32_t i = i0 + lane;
        const float v = i < s1 ? to_f32(l[i]) : 0.0f;
        const uint32_t key = i < s1 ? key_of(v) : 0;
        const u64 w = i < s1 && key >= cut ? weight_of(v, top, inv_t) : 0;
        u64 run = i < s1 && key > cut && w >= least ? w : 0;
        const unsigned tie = __ballot_sync(kFull, i < s1 && key == cut);
        const uint32_t rank = eq_before + __popc(tie & (0xFFFFFFFFu >> (31 - lane)));
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const u64 o = __shfl_up_sync(kFull, run, d);
            if (lane >= d) run += o;
        }
        const unsigned past = __ballot_sync(kFull, before + run + min(rank, ties) * wc > t);
        if (past) {
            if (lane == __ffs(past) - 1) {
                P.ids[row] = (int32_t)i;
                if (P.logprob)
                    P.logprob[row] = greedy ? 0.0f : (float)((double)z_of(v, top, inv_t) - log((double)total * 0x1p-40));
            }
            return;
        }
        before += __shfl_sync(kFull, run, 31);
        eq_before += __popc(tie);
    }
}

}  // namespace
}  // namespace bpe

using namespace bpe;

extern "C" int head_sample(bpe_ctx *ctx, const void *d_logits, uint64_t stride, int type, uint32_t n_rows, uint32_t n_tok,
                           const float *d_u, const head_filters *filters, int32_t *d_ids_out, float *d_logprob_out) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    if (!head_type_ok(type)) return fail(ctx, BPE_ERR_INVALID_ARG, "head_sample: unknown element type");
    if (n_tok == 0 || n_tok > BPE_HEAD_MAX_TOKENS)
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_sample: %u tokens outside 1..%u", n_tok, BPE_HEAD_MAX_TOKENS);
    if (n_rows == 0) return BPE_OK;
    if (n_rows > 0x7FFFFFFFu) return fail(ctx, BPE_ERR_INVALID_ARG, "head_sample: %u rows", n_rows);
    if (!d_logits || !d_u || !d_ids_out) return fail(ctx, BPE_ERR_INVALID_ARG, "head_sample: null pointer");
    if (n_rows > 1 && stride < n_tok) return fail(ctx, BPE_ERR_INVALID_ARG, "head_sample: the row stride is below n_tok");
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    const head_filters none{1.0f, 0, 1.0f, 0.0f, nullptr, nullptr, nullptr, nullptr};
    SampleParams P{d_logits, stride, n_tok, d_u, filters ? *filters : none, d_ids_out, d_logprob_out};
    if (type == BPE_F32)
        k_head_sample<float><<<n_rows, kSampThreads, 0, ctx->stream>>>(P);
    else if (type == BPE_BF16)
        k_head_sample<__nv_bfloat16><<<n_rows, kSampThreads, 0, ctx->stream>>>(P);
    else
        k_head_sample<__half><<<n_rows, kSampThreads, 0, ctx->stream>>>(P);
    BPE_CUDA(ctx, cudaGetLastError(), "head_sample launch");
    return BPE_OK;
}
