// e4m3 codes with a scale per block of 128: tokens (128 values of a row, pwq_quantize_tokens_fp8) and
// weights (128 x 128, pwq_quantize_blocks_fp8), the operands of pwq_quantized_matmul_fp8.
//
// Per block with largest magnitude top:
//   float32 scales: s = float32(top / 448), s below 2^-120 counts as 0
//   e8m0 scales:    s = 2^n, n the least integer with top <= 448 2^n, not below -127
//   code = the e4m3 value nearest to y / s, ties to even; a value that is not finite makes s NaN,
//   and s = 0 or NaN makes every code 0.
//
// The code is that of the exact quotient.  y times a reciprocal is off by up to 2^-23 of itself, which
// matters only next to the middle of two e4m3 values, so each value is converted twice, with the
// reciprocal 2^-22 too small and too large: two multiplies and one conversion of a pair, which keeps
// up with memory where a division would not.  The rounding is monotone, so equal codes are right;
// where they differ, by one step then, the sign of y - (middle) s decides, exact in float64.  Powers
// of two divide exactly.
//
// One pass: a block stays in registers between its maximum and its codes.
#include "../../include/pwq.h"
#include "fp8.h"
#include "tokens.h"

namespace pwq {

namespace {

struct F8QuantArgs {
    const void* X;                 // tokens x d, or matrices of m x d
    uint8_t* Q;
    void* S;                       // float32 or e8m0
    int64_t ldx, ldq, lds, T;      // tokens, or rows of a matrix; lds: the tokens' scales' pitch
    int64_t stride;                // between matrices
    int64_t tiles, tiles_t, tiles_g;
    int64_t mats;
    int d, groups, tshift;
};

// Rotation within rows of 16 lanes
template <int N>
__device__ __forceinline__ float row_ror(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, false));
}
// The largest over 16 lanes, NaN if one is, in all of them
__device__ __forceinline__ float max16(float v) {
    v = max_nan(v, row_ror<8>(v));
    v = max_nan(v, row_ror<4>(v));
    v = max_nan(v, row_ror<2>(v));
    return max_nan(v, row_ror<1>(v));
}
template <int XT>
__device__ __forceinline__ float top8(const Raw<XT>& x) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max_nan(m, __builtin_fabsf(x.get(e)));
    return m;
}

struct F8Scale {
    float s, inv;                  // inv = 1 / s rounded once, 0 where every code is 0
    uint8_t e8;
};
template <bool E8>
__device__ __forceinline__ F8Scale f8_scale(float top) {
    F8Scale r{0.f, 0.f, 0};
    const bool finite = __builtin_isfinite(top);
    if constexpr (E8) {
        int n = __builtin_amdgcn_frexp_expf(top) - 9 + (__builtin_amdgcn_frexp_mantf(top) > 0.875f ? 1 : 0);
        n = n > -127 && top > 0.f ? n : -127;
        r.e8 = finite ? (uint8_t)(n + 127) : 255;
        r.inv = finite ? __builtin_ldexpf(1.f, -n) : 0.f;
    } else {
        r.s = top / F8_TOP;
        if (r.s < F8_TINY) r.s = 0.f;
        r.inv = finite && r.s > 0.f ? 1.f / r.s : 0.f;
        if (!finite) r.s = __builtin_nanf("");
    }
    return r;
}

// four values' codes, the first in the low byte
__device__ __forceinline__ uint32_t f8_pack(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return (uint32_t)w;
}

// the code of y between two neighbours lo and hi (of y's sign, or zeros)
__device__ __forceinline__ uint32_t f8_between(float y, float s, uint32_t lo, uint32_t hi) {
    const double mid = 0.5 * ((double)__builtin_amdgcn_cvt_f32_fp8((int)(lo & 127u), 0) +
                              (double)__builtin_amdgcn_cvt_f32_fp8((int)(hi & 127u), 0));
    const double r = (double)__builtin_fabsf(y) - mid * (double)s;
    return r > 0.0 || (r == 0.0 && (lo & 1u)) ? hi : lo;
}

// eight codes
template <int XT, bool E8>
__device__ __forceinline__ void f8_codes(uint32_t (&w)[2], const Raw<XT>& x, const F8Scale& s) {
    if constexpr (E8) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            w[k] = f8_pack(x.get(4 * k) * s.inv, x.get(4 * k + 1) * s.inv, x.get(4 * k + 2) * s.inv, x.get(4 * k + 3) * s.inv);
    } else {
        const float lo = s.inv * (1.f - 0x1p-22f), hi = s.inv * (1.f + 0x1p-22f);
        uint32_t v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            w[k] = f8_pack(x.get(4 * k) * lo, x.get(4 * k + 1) * lo, x.get(4 * k + 2) * lo, x.get(4 * k + 3) * lo);
            v[k] = f8_pack(x.get(4 * k) * hi, x.get(4 * k + 1) * hi, x.get(4 * k + 2) * hi, x.get(4 * k + 3) * hi);
        }
        if (w[0] != v[0] || w[1] != v[1]) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t u = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t a = (w[k] >> (8 * e)) & 255u, b = (v[k] >> (8 * e)) & 255u;
                    u |= (a == b ? a : f8_between(x.get(4 * k + e), s.s, a, b)) << (8 * e);
                }
                w[k] = u;
            }
        }
    }
    if (s.inv == 0.f) w[0] = w[1] = 0u;                   // NaN among the values, or -0
}

template <int AL>
__device__ __forceinline__ void f8_store(uint8_t* q, int col, int d, const uint32_t (&w)[2]) {
    if constexpr (AL == ROWS_VEC) {
        *(uint2*)(q + col) = make_uint2(w[0], w[1]);
    } else if (col + 8 <= d) {
        __builtin_memcpy(q + col, w, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (col + e < d) q[col + e] = (uint8_t)(w[e / 4] >> (8 * (e & 3)));
    }
}

// a / b, in 32 bits where they fit
__device__ __forceinline__ int64_t f8q_div(int64_t a, int64_t b) {
    return ((uint64_t)(a | b) >> 32) ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// ------------------------------------------------------------------ tokens
// 16 lanes hold a token's 128 values, eight each.  A workgroup takes 2^tshift tokens (16, fewer where
// there are fewer) by 16 / 2^tshift groups in U turns, so that the scales of 16 tokens are written in
// one piece and all loads are under way before the first maximum.  Workgroups go through a row's groups
// first: through the tokens first 8192 x 8192 takes 49 us in place of 44 (rows 16 KB apart meet in the
// same memory channels).
//
// U is 1 where workgroups are few or a row is one turn (16 x 8192 2.9 us, 3.8 with two and 5.0 with four
// turns; 100000 x 128 12.9, 13.8 and 15.5); else 2 for float32 scales on aligned rows and 4 otherwise
// (bfloat16: 4096 x 28672 72.5 us with two, 74.6 with four and 83.5 with one; 4096 x 28671 89, 79 and 93;
// float16, powers of two: 4096 x 28672 66.5, 63.4 and 66.6).
constexpr int64_t F8Q_FEW = 16 * 256;

template <int XT, int AL, bool E8, int U>
__global__ __launch_bounds__(256) void f8_tokens_kernel(F8QuantArgs a) {
    const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int wide = 16 >> a.tshift;                      // groups side by side
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const int64_t tt = f8q_div(tile, a.tiles_g);
        const int64_t t = (tt << a.tshift) + (sub & ((1 << a.tshift) - 1));
        const int g0 = (int)(tile - tt * a.tiles_g) * (wide * U) + (sub >> a.tshift);
        const char* row = (const char*)a.X + (t < a.T ? t : a.T - 1) * a.ldx * Raw<XT>::SIZE;
        Raw<XT> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t col = (int64_t)(g0 + u * wide) * F8_B + 8 * l;
            x[u].template fetch<AL>(row, (int)(col < a.d ? col : a.d), a.d);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = g0 + u * wide;
            const int64_t col64 = (int64_t)g * F8_B + 8 * l;
            const int col = (int)(col64 < a.d ? col64 : a.d);
            x[u].template settle<AL>(col, a.d);
            if (col >= a.d) x[u].zero();
            const F8Scale s = f8_scale<E8>(max16(top8(x[u])));
            if (t >= a.T || col >= a.d) continue;
            uint32_t w[2];
            f8_codes<XT, E8>(w, x[u], s);
            f8_store<AL>(a.Q + t * a.ldq, col, a.d, w);
            if (l == 0) {
                if (E8) ((uint8_t*)a.S)[g * a.lds + t] = s.e8;
                else ((float*)a.S)[g * a.lds + t] = s.s;
            }
        }
    }
}

// ------------------------------------------------------------------ weights
// A workgroup holds a block of 128 x 128, 64 values a thread.  Memory bounds it: 8192 x 28672 float16 141
// us (5.0 TB/s), float32 217 (5.4); rows of odd length 8191 x 8191 bfloat16 58, where 8192 x 8192 takes 45: a
// row of a block shares a line of 128 bytes with the next block, whose workgroup is on another XCD, and both
// read it (201 MB for 134).
template <int XT, int AL, bool E8>
__global__ __launch_bounds__(256) void f8_blocks_kernel(F8QuantArgs a) {
    __shared__ float slot[2][4];
    const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;
    int par = 0;
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x, par ^= 1) {
        const int64_t rest = f8q_div(tile, a.groups), mat = f8q_div(rest, a.tiles_t), ob = rest - mat * a.tiles_t;
        const int g = (int)(tile - rest * a.groups);
        const char* base = (const char*)a.X + mat * a.stride * Raw<XT>::SIZE;
        const int col = g * F8_B + 8 * l;                 // d is below 2^30 + 128
        Raw<XT> x[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int64_t r = ob * F8_B + 16 * p + sub;
            x[p].template fetch<AL>(base + (r < a.T ? r : a.T - 1) * a.ldx * Raw<XT>::SIZE, col < a.d ? col : a.d, a.d);
        }
        float top = 0.f;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            x[p].template settle<AL>(col, a.d);
            if (col >= a.d) x[p].zero();
            top = max_nan(top, top8(x[p]));               // rows past the end repeat the last one
        }
        const F8Scale s = f8_scale<E8>(row_reduce<256>(max16(top), slot[par], [](float u, float v) { return max_nan(u, v); }));
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int64_t r = ob * F8_B + 16 * p + sub;
            if (r >= a.T || col >= a.d) continue;
            uint32_t w[2];
            f8_codes<XT, E8>(w, x[p], s);
            f8_store<AL>(a.Q + (mat * a.T + r) * a.d, col, a.d, w);
        }
        if (threadIdx.x == 0) {
            const int64_t i = (mat * a.tiles_t + ob) * a.groups + g;
            if (E8) ((uint8_t*)a.S)[i] = s.e8;
            else ((float*)a.S)[i] = s.s;
        }
    }
}

// ------------------------------------------------------------------ launches
constexpr int64_t F8Q_MAX_GROUPS = 1 << 20;               // tiles past this are taken by the kernel's loop

template <int XT, int AL, bool E8, int U>
void f8q_tokens(F8QuantArgs a, hipStream_t s) {
    a.tiles_g = cdiv(a.groups, (16 >> a.tshift) * U);
    a.tiles = a.tiles_t * a.tiles_g;
    const dim3 grid((unsigned)(a.tiles < F8Q_MAX_GROUPS ? a.tiles : F8Q_MAX_GROUPS));
    hipLaunchKernelGGL((f8_tokens_kernel<XT, AL, E8, U>), grid, dim3(256), 0, s, a);
}
template <int XT, int AL, bool E8, bool TOKENS>
void f8q_go(const F8QuantArgs& a, hipStream_t s) {
    if constexpr (TOKENS) {
        const int64_t turns = cdiv(a.groups, 16 >> a.tshift);
        if (AL == ROWS_SHORT || turns == 1 || a.tiles_t * turns <= F8Q_FEW) f8q_tokens<XT, AL, E8, 1>(a, s);
        else if constexpr (AL != ROWS_SHORT) f8q_tokens<XT, AL, E8, AL == ROWS_VEC && !E8 ? 2 : 4>(a, s);
    } else {
        const dim3 grid((unsigned)(a.tiles < F8Q_MAX_GROUPS ? a.tiles : F8Q_MAX_GROUPS));
        hipLaunchKernelGGL((f8_blocks_kernel<XT, AL, E8>), grid, dim3(256), 0, s, a);
    }
}
template <int XT, bool TOKENS>
void f8q_rows(const F8QuantArgs& a, bool e8, hipStream_t s) {
    const bool vec = a.d % 8 == 0 && a.ldx % 8 == 0 && a.ldq % 8 == 0 && a.stride % 8 == 0 && aligned(a.X, 16) && aligned(a.Q, 8);
    if (vec) (e8 ? f8q_go<XT, ROWS_VEC, true, TOKENS>(a, s) : f8q_go<XT, ROWS_VEC, false, TOKENS>(a, s));
    else if (a.d >= 8) (e8 ? f8q_go<XT, ROWS_ANY, true, TOKENS>(a, s) : f8q_go<XT, ROWS_ANY, false, TOKENS>(a, s));
    else (e8 ? f8q_go<XT, ROWS_SHORT, true, TOKENS>(a, s) : f8q_go<XT, ROWS_SHORT, false, TOKENS>(a, s));
}
template <bool TOKENS>
hipError_t f8q_run(const F8QuantArgs& a, int x_dtype, bool e8, hipStream_t s) {
    if (x_dtype == 0) f8q_rows<0, TOKENS>(a, e8, s);
    else if (x_dtype == 1) f8q_rows<1, TOKENS>(a, e8, s);
    else f8q_rows<2, TOKENS>(a, e8, s);
    return hipGetLastError();
}

}  // namespace

hipError_t f8_tokens_launch(const void* X, int x_dtype, int64_t T, int64_t d, int64_t ldx, bool e8, uint8_t* Q, int64_t ldq,
                            void* S, int64_t lds, hipStream_t s) {
    F8QuantArgs a{};
    a.X = X; a.Q = Q; a.S = S; a.ldx = ldx; a.ldq = ldq; a.lds = lds; a.T = T; a.d = (int)d;
    a.groups = (int)cdiv(d, F8_B);
    while (a.tshift < 4 && (1 << a.tshift) < T) ++a.tshift;
    a.tiles_t = cdiv(T, 1 << a.tshift);
    return f8q_run<true>(a, x_dtype, e8, s);
}

hipError_t f8_blocks_launch(const void* W, int w_dtype, int64_t mats, int64_t m, int64_t d, int64_t ldw, int64_t stride,
                            bool e8, uint8_t* Q, void* S, hipStream_t s) {
    F8QuantArgs a{};
    a.X = W; a.Q = Q; a.S = S; a.ldx = ldw; a.ldq = d; a.stride = mats > 1 ? stride : 0; a.T = m; a.d = (int)d;
    a.groups = (int)cdiv(d, F8_B);
    a.tiles_t = cdiv(m, F8_B);
    a.tiles = mats * a.tiles_t * a.groups;
    return f8q_run<false>(a, w_dtype, e8, s);
}

}  // namespace pwq
