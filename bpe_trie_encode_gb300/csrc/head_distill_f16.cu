// head_distill_f16.cu -- head_distill's kernels for logits of this type.
#include "head_distill.cuh"

namespace bpe {
int distill_f16(bpe_ctx *ctx, const DistillParams &P, uint32_t n_rows) { return launch<__half>(ctx, P, n_rows); }
}  // namespace bpe
