// head_distill_bf16.cu -- head_distill's kernels for logits of this type.
#include "head_distill.cuh"

namespace bpe {
int distill_bf16(bpe_ctx *ctx, const DistillParams &P, uint32_t n_rows) { return launch<__nv_bfloat16>(ctx, P, n_rows); }
}  // namespace bpe
