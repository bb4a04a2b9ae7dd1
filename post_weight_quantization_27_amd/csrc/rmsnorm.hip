// Root-mean-square norm with the residual's addition and 8-bit codes (pwq_rms_norm_quantize); the
// kernels are in tokens.h.
#include "tokens.h"

namespace pwq {

hipError_t rms_norm_launch(const void* X, int x_dtype, int64_t T, int64_t d, int64_t ldx, const void* R, int64_t ldr,
                           const void* G, int g_dtype, double eps, void* H, int64_t ldh, int8_t* Q, int64_t ldq, float* S,
                           int32_t* sums, void* Y, int y_dtype, int64_t ldy, hipStream_t s) {
    TokArgs a{};
    a.X = X; a.ldx = ldx; a.T = T; a.d = (int)d; a.R = R; a.ldr = ldr; a.G = G; a.g_dtype = g_dtype; a.eps = eps;
    a.H = H; a.ldh = ldh; a.Q = Q; a.ldq = ldq; a.S = S; a.sums = sums; a.Y = Y; a.y_dtype = y_dtype; a.ldy = ldy;
    const bool vec = d % 8 == 0 && rows16(X, ldx, x_dtype) && rows16(R, ldr, x_dtype) && rows16(H, ldh, x_dtype) &&
                     rows16(G, 8, g_dtype) && rows16(Y, ldy, y_dtype) && (!Q || (aligned(Q, 8) && ldq % 8 == 0));
    if (x_dtype != 0 && (!G || g_dtype != 0)) return tok_type<TOK_NORM16>(a, x_dtype, vec, s);
    return tok_type<TOK_NORM64>(a, x_dtype, vec, s);
}

}  // namespace pwq
