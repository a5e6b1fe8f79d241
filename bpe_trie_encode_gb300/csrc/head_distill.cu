// head_distill.cu -- divergence of rows of logits from a teacher's top
// alternatives, and its gradient in the same call.
#include "head_row.cuh"

namespace bpe {
namespace {

constexpr int kMost = (int)BPE_HEAD_MAX_TOP;   // alternatives that a teacher lists
constexpr size_t kMostShared = 72 * 1024;       // of a CTA: the bits of the most tokens over the largest team
static_assert(kMost <= kRowThreads, "one thread for each");

struct DistillParams {
    RowParams row;
    const int32_t *top_ids;
    const void *top_logprob;
    int top_type;
    uint32_t n_listed;
    int rest;
    float *loss;
    float grad;
    const float *d_grad;
    void *out;
    uint64_t out_stride;
};

struct DistillShared {
    TeamShared team;
    uint32_t id[kMost];        // ~0: none
    float q[kMost], v[kMost];  // the entry's q, its token's logit
    uint32_t bits[1];          // a bit for each place of the CTA's vectors: listed
};

// What the row's listed entries come to.
struct Listed { float q_sum, q_log_q; };

// Entries, with their weights and logits, into shared memory.
template <typename T>
__device__ __forceinline__ Listed read_entries(DistillShared &S, Team<false> &cta, const DistillParams &P, uint32_t r, const RowView<T> &row) {
    const uint32_t i = threadIdx.x;
    uint32_t id = ~0u;
    float t = -INFINITY, v = -INFINITY;
    if (i < P.n_listed) {
        const uint64_t at = (uint64_t)r * P.n_listed + i;
        id = (uint32_t)P.top_ids[at];
        t = P.top_type == BPE_F32    ? ((const float *)P.top_logprob)[at]
            : P.top_type == BPE_BF16 ? to_f32(((const __nv_bfloat16 *)P.top_logprob)[at])
                                     : to_f32(((const __half *)P.top_logprob)[at]);
        if (id >= P.row.n_tok || !(t > -INFINITY)) id = ~0u, t = -INFINITY;
        if (id != ~0u) v = to_f32(row.at[row.shift + id]);
    }
    if (!P.rest) {             // the softmax of the listed values
        const float m = cta.max(t);
        const float z = m > -INFINITY ? z_any(t, m, 1.0f) : -INFINITY;
        const float s = cta.sum(make_float4(expf(z), 0, 0, 0)).x;
        t = z - logf(s);
    }
    const float q = t > -INFINITY ? expf(t) : 0.0f;
    const float4 sum = cta.sum(make_float4(q, q > 0.0f ? q * t : 0.0f, 0, 0));
    if (i < P.n_listed) S.id[i] = id, S.q[i] = q, S.v[i] = v;
    __syncthreads();
    return {sum.x, sum.y};
}

template <typename T, bool kTeam>
__global__ void __launch_bounds__(kRowThreads) k_distill(DistillParams P, uint32_t n_team) {
    constexpr int kVec = RowView<T>::kVec;
    extern __shared__ __align__(16) unsigned char smem[];
    DistillShared &S = *(DistillShared *)smem;
    Team<kTeam> team(S.team, n_team);
    Team<false> cta(S.team, 1);
    team.begin();
    const uint32_t r = kTeam ? blockIdx.x / n_team : blockIdx.x;
    const RowView<T> row(P.row.logits, P.row.stride, r, P.row.n_tok);
    const uint32_t vecs = row.vecs(), share = (vecs + team.size - 1) / team.size;
    const uint32_t lo = min(vecs, team.rank * share), hi = min(vecs, lo + share);
    const float c = P.row.inverse(r);
    const uint32_t k = P.n_listed;

    const Listed listed = read_entries<T>(S, cta, P, r, row);
    if (P.rest) {
        for (uint32_t i = threadIdx.x; i < (share * kVec + 31) / 32; i += kRowThreads) S.bits[i] = 0;
        __syncthreads();
        if (threadIdx.x < k && S.id[threadIdx.x] != ~0u) {
            const uint32_t at = S.id[threadIdx.x] + row.shift;
            if (at >= lo * kVec && at < hi * kVec) atomicOr(&S.bits[(at - lo * kVec) / 32], 1u << ((at - lo * kVec) % 32));
        }
        __syncthreads();
    }
    // the softmax of the tokens that have no entry of their own: of all, where unlisted tokens are no class
    auto load = [&](uint32_t i) {
        uint4 q = row.load(i);
        if (P.rest) {
            const uint32_t at = (i - lo) * kVec, bits = S.bits[at / 32] >> (at % 32);
            for (int e = 0; e < kVec; e++)
                if (bits >> e & 1) RowView<T>::put(q, e, from_f32<T>(-INFINITY));
        }
        return q;
    };
    const Softmax free = softmax_any<T, kTeam>(team, lo, hi, c, load);

    // every entry finds the first of its id, and that one the sum of their q
    bool first = false;
    uint32_t id = ~0u;
    float v = -INFINITY, q_all = 0.0f;
    if (threadIdx.x < k && (id = S.id[threadIdx.x]) != ~0u) {
        first = true;
        v = S.v[threadIdx.x];
        for (uint32_t j = 0; j < k; j++)
            if (S.id[j] == id) q_all += S.q[j], first &= j >= threadIdx.x;
    }
    // the whole row's softmax: m, s, relative to which the unlisted tokens' is
    float m = free.m, s = free.s, to_all = 1.0f;
    if (P.rest) {
        m = fmaxf(cta.max(first ? v == v ? v : -INFINITY : -INFINITY), free.m);
        if (m > -INFINITY) {
            to_all = free.m > -INFINITY ? expf(z_any(free.m, m, c)) : 0.0f;
            s = free.s * to_all + cta.sum(make_float4(first ? expf(z_any(v, m, c)) : 0.0f, 0, 0, 0)).x;
        }
    }
    const bool none = m == -INFINITY;
    const float log_s = logf(s);
    const float z = none ? -INFINITY : z_any(v, m, c);
    float term = 0.0f;
    if (threadIdx.x < k && S.q[threadIdx.x] > 0.0f) term = S.q[threadIdx.x] * (z - log_s);
    const float cross = cta.sum(make_float4(term, 0, 0, 0)).x;
    const float q_rest = P.rest && free.m > -INFINITY ? fmaxf(0.0f, 1.0f - listed.q_sum) : 0.0f, q_total = listed.q_sum + q_rest;
    if (threadIdx.x == 0 && team.rank == 0) {
        float loss = listed.q_log_q - cross;
        if (q_rest > 0.0f) {
            loss += q_rest * (logf(q_rest) - (z_any(free.m, m, c) + logf(free.s) - log_s));
        }
        P.loss[r] = none ? (q_total > 0.0f ? INFINITY : 0.0f) : loss;
    }
    if (!P.out) return;

    const RowView<T> out(P.out, P.out_stride, r, P.row.n_tok);
    const bool zero = none || c == INFINITY;
    const float g = zero ? 0.0f : c * (P.d_grad ? P.d_grad[r] : P.grad);
    const float of_free = q_total / s * to_all - (q_rest > 0.0f ? q_rest / free.s : 0.0f);
    __syncthreads();
    const uint32_t t0 = lo * kVec, t1 = hi * kVec;   // places of the CTA's vectors
    for (uint32_t at = t0 + threadIdx.x; at < t1; at += kRowThreads)
        if (at >= row.shift && at < row.end) {
            const float x = zero || free.m == -INFINITY ? 0.0f : expf(z_any(to_f32(row.at[at]), free.m, c));
            out.at[out.shift + at - row.shift] = from_f32<T>(zero ? 0.0f : g * (x * of_free));
        }
    __syncthreads();
    if (first && id + row.shift >= t0 && id + row.shift < t1)
        out.at[out.shift + id] = from_f32<T>(zero ? 0.0f : g * (q_total * expf(z - log_s) - q_all));
}

template <typename T, bool kTeam> int launch_team(bpe_ctx *ctx, const DistillParams &P, uint32_t n_rows, uint32_t team, size_t smem) {
    auto k = k_distill<T, kTeam>;
    static std::atomic<uint64_t> devices{0};
    BPE_CUDA(ctx, allow_shared(k, ctx->device, kMostShared, devices), "head_distill");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n_rows * team);
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = ctx->stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {team, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = kTeam ? 1 : 0;
    BPE_CUDA(ctx, cudaLaunchKernelEx(&cfg, k, P, team), "head_distill launch");
    return BPE_OK;
}

template <typename T> int launch(bpe_ctx *ctx, const DistillParams &P, uint32_t n_rows) {
    constexpr uint32_t kVec = RowView<T>::kVec;
    const uint32_t vecs = (P.row.n_tok + kVec - 1) / kVec + 1;   // of a row that starts anywhere
    auto shared = [&](uint32_t team) {
        return sizeof(DistillShared) + (P.rest ? (size_t)((vecs + team - 1) / team * kVec + 31) / 32 * 4 : 0);
    };
    uint32_t team = 1;
    while (team < kMaxTeam && shared(team) > kMostShared) team *= 2;
    return team > 1 ? launch_team<T, true>(ctx, P, n_rows, team, shared(team)) : launch_team<T, false>(ctx, P, n_rows, 1, shared(1));
}

}  // namespace
}  // namespace bpe

using namespace bpe;

extern "C" int head_distill(bpe_ctx *ctx, const void *d_logits, uint64_t stride, int type, uint32_t n_rows, uint32_t n_tok,
                            const int32_t *d_top_ids, const void *d_top_logprob, int top_type, uint32_t n_listed, int rest,
                            float temperature, const float *d_temperature, float *d_loss_out, float grad, const float *d_grad,
                            void *d_grad_out, uint64_t grad_stride) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    const char *const name = "head_distill";
    if (const int rc = head_row_check(ctx, name, d_logits, stride, type, n_rows, n_tok)) return rc;
    if (!head_type_ok(top_type)) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: unknown element type", name);
    if (n_listed == 0 || n_listed > BPE_HEAD_MAX_TOP)
        return fail(ctx, BPE_ERR_INVALID_ARG, "%s: %u listed tokens outside 1..%u", name, n_listed, BPE_HEAD_MAX_TOP);
    if (n_rows == 0) return BPE_OK;
    if (!d_top_ids || !d_top_logprob || !d_loss_out) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (d_grad_out)
        if (const int rc = head_grad_check(ctx, name, d_logits, stride, type, n_rows, n_tok, d_grad_out, grad_stride)) return rc;
    if (const int rc = head_report(ctx)) return rc;
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    const DistillParams P{{d_logits, stride, n_tok, temperature, d_temperature}, d_top_ids, d_top_logprob, top_type, n_listed,
                          rest, d_loss_out, grad, d_grad, d_grad_out, grad_stride};
    return type == BPE_F32    ? launch<float>(ctx, P, n_rows)
           : type == BPE_BF16 ? launch<__nv_bfloat16>(ctx, P, n_rows)
                              : launch<__half>(ctx, P, n_rows);
}
