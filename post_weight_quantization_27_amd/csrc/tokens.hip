// 8-bit codes of activations per token (pwq_quantize_tokens); the kernels are in tokens.h.
#include "tokens.h"

namespace pwq {

hipError_t tok_quant_launch(const void* X, int x_dtype, int64_t T, int64_t d, int64_t ldx, const float* chan, int8_t* Q,
                            int64_t ldq, float* S, int32_t* sums, hipStream_t s) {
    TokArgs a{};
    a.X = X; a.ldx = ldx; a.T = T; a.d = (int)d; a.chan = chan;
    a.Q = Q; a.ldq = ldq; a.S = S; a.sums = sums;
    const bool vec = d % 8 == 0 && rows16(X, ldx, x_dtype) && rows16(chan, 4, 0) && aligned(Q, 8) && ldq % 8 == 0;
    return chan ? tok_type<TOK_CHAN>(a, x_dtype, vec, s) : tok_type<TOK_PLAIN>(a, x_dtype, vec, s);
}

}  // namespace pwq
