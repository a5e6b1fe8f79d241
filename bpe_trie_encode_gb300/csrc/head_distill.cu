// head_distill.cu -- the entry point of head_distill (head_distill.cuh).
#include "head_distill.cuh"

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
    return type == BPE_F32    ? distill_f32(ctx, P, n_rows)
           : type == BPE_BF16 ? distill_bf16(ctx, P, n_rows)
                              : distill_f16(ctx, P, n_rows);
}
