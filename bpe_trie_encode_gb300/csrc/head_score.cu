// head_score.cu -- log-probabilities of given ids, with the entropy and the top
// alternatives of each row of logits, and the gradient of both.
#include "head_row.cuh"

namespace bpe {
namespace {

constexpr int kTop = (int)BPE_HEAD_MAX_TOP;
constexpr int kList = 1024;                // tokens that may be among the alternatives

struct ScoreParams {
    RowParams row;
    const int32_t *ids;
    uint32_t n_top;
    float *logprob, *entropy;
    int32_t *top_ids;
    float *top_logprob;
    float *norm;
};

struct ScoreShared {
    TeamShared team;
    uint32_t list_n, scan[kRowWarps];
    u64 list[kList];                       // key of the logit, then the id from above, so that the larger comes first
    u64 best[kTop];                        // in order
};

__device__ __forceinline__ u64 entry_of(uint32_t key, uint32_t id) { return (u64)key << 32 | (uint32_t)~id; }

// The alternatives in S.list, at most k of this CTA's, for any logits: the key of the k-th largest is found by bits, two
// a pass; those above it are listed, and as many of its equals, in order of ids, as there is room for.
template <typename T, bool kTeam>
__device__ __noinline__ void list_any(ScoreShared &S, Team<kTeam> &team, const RowView<T> &row, uint32_t lo, uint32_t hi, uint32_t k) {
    constexpr int kVec = RowView<T>::kVec, kShift = Bits<T>::kShift, kBits = (32 - kShift + 1) & ~1;
    uint32_t some = 0;
    for (uint32_t i = lo + threadIdx.x; i < hi; i += kRowThreads) {
        float v[kVec];
        unpack(row.load(i), v, T());
#pragma unroll
        for (int e = 0; e < kVec; e++) some += v[e] > -INFINITY;
    }
    const float valid = team.sum(make_float4(some, 0, 0, 0)).x;   // counts up to 2^22 are exact in 32 bits
    const float want = fminf((float)k, valid);
    if (threadIdx.x == 0) S.list_n = 0;
    __syncthreads();
    if (want == 0.0f) return;
    uint32_t cut = 0;
    for (int bit = kBits - 2; bit >= 0; bit -= 2) {
        uint32_t n1 = 0, n2 = 0, n3 = 0;
        for (uint32_t i = lo + threadIdx.x; i < hi; i += kRowThreads) {
            float v[kVec];
            unpack(row.load(i), v, T());
#pragma unroll
            for (int e = 0; e < kVec; e++) {
                const uint32_t key = key_of(v[e]) >> kShift;
                n1 += key >= (cut | 1u << bit), n2 += key >= (cut | 2u << bit), n3 += key >= (cut | 3u << bit);
            }
        }
        const float4 n = team.sum(make_float4(n1, n2, n3, 0));
        cut |= (n.z >= want ? 3u : n.y >= want ? 2u : n.x >= want ? 1u : 0u) << bit;
    }
    uint32_t above = 0, equal = 0;
    for (uint32_t i = lo + threadIdx.x; i < hi; i += kRowThreads) {
        float v[kVec];
        unpack(row.load(i), v, T());
#pragma unroll
        for (int e = 0; e < kVec; e++) {
            const uint32_t key = key_of(v[e]);
            if (key >> kShift > cut) S.list[atomicAdd(&S.list_n, 1)] = entry_of(key, i * kVec + e - row.shift), above++;   // fewer than k
            equal += key >> kShift == cut;
        }
    }
    const float4 n = team.sum(make_float4(above, equal, 0, 0));
    uint32_t mine = 0, before = 0;         // equals of this CTA, and of those before it
    if (kTeam) {
        for (uint32_t r = 0; r < team.rank; r++) before += (uint32_t)team.S.slot[team.turn][r].y;
        mine = (uint32_t)team.S.slot[team.turn][team.rank].y;
    } else {
        mine = (uint32_t)n.y;
    }
    const uint32_t need = (uint32_t)(want - n.x);
    const uint32_t quota = min(mine, need > before ? need - before : 0u);
    uint32_t seen = 0;
    for (uint32_t i0 = lo; i0 < hi && seen < quota; i0 += kRowThreads) {
        const uint32_t i = i0 + threadIdx.x;
        float v[kVec];
        uint32_t own = 0;
        if (i < hi) {
            unpack(row.load(i), v, T());
#pragma unroll
            for (int e = 0; e < kVec; e++) own += key_of(v[e]) >> kShift == cut;
        }
        const uint32_t upto = warp_incl_sum(own, team.lane);
        __syncthreads();
        if (team.lane == 31) S.scan[team.warp] = upto;
        __syncthreads();
        uint32_t at = seen + upto - own;
        for (int w = 0; w < kRowWarps; w++) {
            if (w < team.warp) at += S.scan[w];
            seen += S.scan[w];
        }
        if (own) {
#pragma unroll
            for (int e = 0; e < kVec; e++)
                if (key_of(v[e]) >> kShift == cut && at++ < quota)
                    S.list[atomicAdd(&S.list_n, 1)] = entry_of(key_of(v[e]), i * kVec + e - row.shift);
        }
    }
    __syncthreads();
}

// The list's k largest in order, in S.best: each entry's place is the number of larger ones, counted by four threads.
__device__ __forceinline__ uint32_t rank_list(ScoreShared &S, uint32_t k) {
    const uint32_t n = S.list_n, part = threadIdx.x & 3;
    for (uint32_t i0 = 0; i0 < n; i0 += kRowThreads / 4) {
        const uint32_t i = i0 + threadIdx.x / 4;
        const u64 one = S.list[min(i, n - 1)];
        uint32_t place = 0;
        for (uint32_t j = part; j < n; j += 4) place += S.list[j] > one;
        place += __shfl_xor_sync(kFull, place, 1);
        place += __shfl_xor_sync(kFull, place, 2);
        if (i < n && part == 0 && place < k) S.best[place] = one;
    }
    __syncthreads();
    return min(n, k);
}

template <typename T, bool kTeam>
__global__ void __launch_bounds__(kRowThreads) k_logprobs(ScoreParams P, uint32_t n_team) {
    __shared__ ScoreShared S;
    Team<kTeam> team(S.team, n_team);
    const uint32_t r = kTeam ? blockIdx.x / n_team : blockIdx.x;
    const RowView<T> row(P.row.logits, P.row.stride, r, P.row.n_tok);
    const uint32_t vecs = row.vecs(), share = (vecs + team.size - 1) / team.size;
    const uint32_t lo = min(vecs, team.rank * share), hi = min(vecs, lo + share);
    const float c = P.row.inverse(r);
    const uint32_t k = P.top_ids || P.top_logprob ? P.n_top : 0;

    const Softmax all = softmax_any<T, kTeam>(team, lo, hi, c, [&](uint32_t i) { return row.load(i); });
    if (k) list_any<T, kTeam>(S, team, row, lo, hi, k);

    const bool none = all.m == -INFINITY;
    const float log_s = none ? 0.0f : logf(all.s);
    if (threadIdx.x == 0 && team.rank == 0) {
        if (P.norm) P.norm[2 * (uint64_t)r] = all.m, P.norm[2 * (uint64_t)r + 1] = log_s;
        if (P.entropy) P.entropy[r] = none ? 0.0f : log_s - all.sz / all.s;
        if (P.logprob) {
            const int32_t id = P.ids ? P.ids[r] : -1;
            float lp = 0.0f;
            if (id >= 0 && (uint32_t)id < P.row.n_tok) lp = none ? -INFINITY : z_any(to_f32(row.at[row.shift + id]), all.m, c) - log_s;
            P.logprob[r] = lp;
        }
    }
    if (!k) return;
    const uint32_t n = rank_list(S, k);
    for (uint32_t i = threadIdx.x; i < k; i += kRowThreads) {
        const u64 one = S.best[min(i, n)];
        if (P.top_ids) P.top_ids[(uint64_t)r * k + i] = i < n ? (int32_t)~(uint32_t)one : -1;
        if (P.top_logprob) P.top_logprob[(uint64_t)r * k + i] = i < n ? z_any(key_value((uint32_t)(one >> 32)), all.m, c) - log_s : -INFINITY;
    }
}

// ----------------------------------------------------------- gradient ---
struct ScoreGradParams {
    RowParams row;
    const int32_t *ids;
    const float *norm, *grad_logprob, *entropy, *grad_entropy;
    void *out;
    uint64_t out_stride;
};

template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_logprobs_backward(ScoreGradParams P) {
    constexpr int kVec = RowView<T>::kVec;
    const uint32_t r = blockIdx.x;
    const RowView<T> row(P.row.logits, P.row.stride, r, P.row.n_tok), out(P.out, P.out_stride, r, P.row.n_tok);
    const float c = P.row.inverse(r);
    const float2 norm = make_float2(P.norm[2 * (uint64_t)r], P.norm[2 * (uint64_t)r + 1]);
    const int32_t id = P.ids ? P.ids[r] : -1;
    const bool given = id >= 0 && (uint32_t)id < P.row.n_tok;
    const float a = given && P.grad_logprob ? P.grad_logprob[r] : 0.0f, b = P.grad_entropy ? P.grad_entropy[r] : 0.0f;
    const float h = P.grad_entropy ? P.entropy[r] : 0.0f;
    const bool zero = norm.x == -INFINITY || c == INFINITY;
    for (uint32_t j = threadIdx.x; j < P.row.n_tok; j += kRowThreads) {
        const float z = z_any(to_f32(row.at[row.shift + j]), norm.x, c), lp = z - norm.y, p = expf(lp);
        float d = (given && (uint32_t)id == j ? a : 0.0f) - a * p;
        if (p > 0.0f) d -= b * p * (lp + h);
        out.at[out.shift + j] = from_f32<T>(zero ? 0.0f : c * d);
    }
}

template <typename T> int launch_logprobs(bpe_ctx *ctx, const ScoreParams &P, uint32_t n_rows) {
    k_logprobs<T, false><<<n_rows, kRowThreads, 0, ctx->stream>>>(P, 1);
    BPE_CUDA(ctx, cudaGetLastError(), "head_logprobs launch");
    return BPE_OK;
}

template <typename T> int launch_backward(bpe_ctx *ctx, const ScoreGradParams &P, uint32_t n_rows) {
    k_logprobs_backward<T><<<n_rows, kRowThreads, 0, ctx->stream>>>(P);
    BPE_CUDA(ctx, cudaGetLastError(), "head_logprobs_backward launch");
    return BPE_OK;
}

}  // namespace

int head_row_check(bpe_ctx *ctx, const char *name, const void *d_logits, uint64_t stride, int type, uint32_t n_rows,
                   uint32_t n_tok) {
    if (!head_type_ok(type)) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: unknown element type", name);
    if (n_tok == 0 || n_tok > BPE_HEAD_MAX_TOKENS)
        return fail(ctx, BPE_ERR_INVALID_ARG, "%s: %u tokens outside 1..%u", name, n_tok, BPE_HEAD_MAX_TOKENS);
    if (n_rows > 0x7FFFFFFFu) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: %u rows", name, n_rows);
    if (n_rows && !d_logits) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (n_rows && (uintptr_t)d_logits % head_type_size(type))
        return fail(ctx, BPE_ERR_INVALID_ARG, "%s: logits that do not start on an element", name);
    if (n_rows > 1 && stride < n_tok) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: the row stride is below n_tok", name);
    return BPE_OK;
}

int head_grad_check(bpe_ctx *ctx, const char *name, const void *d_logits, uint64_t stride, int type, uint32_t n_rows,
                    uint32_t n_tok, const void *d_grad, uint64_t grad_stride) {
    if (n_rows == 0) return BPE_OK;
    if (!d_grad) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: null pointer", name);
    const size_t e = head_type_size(type);
    if ((uintptr_t)d_grad % e) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: a gradient that does not start on an element", name);
    if (n_rows > 1 && grad_stride < n_tok)
        return fail(ctx, BPE_ERR_INVALID_ARG, "%s: the gradient's row stride is below n_tok", name);
    // The rows of the two may interleave (columns of one buffer), but no row's bytes may be another's: with equal strides the
    // distance of the two within a row's period decides; with others the whole ranges must be apart.
    const uintptr_t x = (uintptr_t)d_logits, y = (uintptr_t)d_grad;
    if (x == y && (n_rows == 1 || stride == grad_stride)) return BPE_OK;
    const uint64_t xs = n_rows > 1 ? stride : n_tok, ys = n_rows > 1 ? grad_stride : n_tok;
    const uintptr_t xe = x + ((uint64_t)(n_rows - 1) * xs + n_tok) * e, ye = y + ((uint64_t)(n_rows - 1) * ys + n_tok) * e;
    bool apart = xe <= y || ye <= x;
    if (!apart && n_rows > 1 && xs == ys) {
        const uint64_t period = xs * e, off = y >= x ? (y - x) % period : (period - (x - y) % period) % period;
        apart = off >= (uint64_t)n_tok * e && off + (uint64_t)n_tok * e <= period;
    }
    if (!apart) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: the gradient overlaps the logits, and is not the logits themselves", name);
    return BPE_OK;
}

}  // namespace bpe

using namespace bpe;

extern "C" int head_logprobs(bpe_ctx *ctx, const void *d_logits, uint64_t stride, int type, uint32_t n_rows, uint32_t n_tok,
                             const int32_t *d_ids, float temperature, const float *d_temperature, uint32_t n_top,
                             float *d_logprob_out, float *d_entropy_out, int32_t *d_top_ids_out, float *d_top_logprob_out,
                             float *d_norm_out) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    if (const int rc = head_row_check(ctx, "head_logprobs", d_logits, stride, type, n_rows, n_tok)) return rc;
    if (n_top > BPE_HEAD_MAX_TOP)
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_logprobs: %u alternatives, at most %u", n_top, BPE_HEAD_MAX_TOP);
    if (n_rows == 0) return BPE_OK;
    if (d_logprob_out && !d_ids) return fail(ctx, BPE_ERR_INVALID_ARG, "head_logprobs: log-probabilities without ids");
    if (const int rc = head_report(ctx)) return rc;
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    const ScoreParams P{{d_logits, stride, n_tok, temperature, d_temperature}, d_ids, n_top, d_logprob_out, d_entropy_out,
                        d_top_ids_out, d_top_logprob_out, d_norm_out};
    return type == BPE_F32    ? launch_logprobs<float>(ctx, P, n_rows)
           : type == BPE_BF16 ? launch_logprobs<__nv_bfloat16>(ctx, P, n_rows)
                              : launch_logprobs<__half>(ctx, P, n_rows);
}

extern "C" int head_logprobs_backward(bpe_ctx *ctx, const void *d_logits, uint64_t stride, int type, uint32_t n_rows,
                                      uint32_t n_tok, const int32_t *d_ids, float temperature, const float *d_temperature,
                                      const float *d_norm, const float *d_grad_logprob, const float *d_entropy,
                                      const float *d_grad_entropy, void *d_grad_out, uint64_t grad_stride) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    const char *const name = "head_logprobs_backward";
    if (const int rc = head_row_check(ctx, name, d_logits, stride, type, n_rows, n_tok)) return rc;
    if (const int rc = head_grad_check(ctx, name, d_logits, stride, type, n_rows, n_tok, d_grad_out, grad_stride)) return rc;
    if (n_rows == 0) return BPE_OK;
    if (!d_norm) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (d_grad_logprob && !d_ids) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: a gradient of log-probabilities without ids", name);
    if (d_grad_entropy && !d_entropy) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: a gradient of entropies without them", name);
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    const ScoreGradParams P{{d_logits, stride, n_tok, temperature, d_temperature}, d_ids, d_norm, d_grad_logprob,
                            d_entropy, d_grad_entropy, d_grad_out, grad_stride};
    return type == BPE_F32    ? launch_backward<float>(ctx, P, n_rows)
           : type == BPE_BF16 ? launch_backward<__nv_bfloat16>(ctx, P, n_rows)
                              : launch_backward<__half>(ctx, P, n_rows);
}
