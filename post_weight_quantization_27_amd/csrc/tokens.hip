// 8-bit codes of activations, one symmetric scale per token, alone (pwq_quantize_tokens) and
// fused with the root-mean-square norm and the residual's addition (pwq_rms_norm_quantize):
// the X operand of the int8 product (pwq_quantized_matmul_int8).
//
// Per row of values y (float64 below means: exact to 2^-53, far finer than any level border):
//   s = float32(max |y| / 127); s below 2^-120 counts as 0, a value that is not finite makes s NaN;
//   code = nearest integer to y / s, ties to even (s = 0 or NaN: code 0).
// Token quantizer: y = x, or the float32 quotient x / c with a scale c per channel.
// Norm: h = x + r rounded once to x's type, y = h g / sqrt(mean(h^2) + eps).  Since
// max |y| = rstd max |h g|, the sum of squares and the largest |h g| come out of ONE pass over
// the row and one reduction; the codes are then nearest(h g (rstd / s)).
//
// The arithmetic is float64: v_fma_f64 runs at the full float32 rate on this chip, h g and h^2
// of 16-bit inputs are exact in it, and a code next to a border between two levels comes out as
// the 64-bit definition says, whatever the order of the sum.  The nearest integer is one fma
// with 1.5 * 2^52 added, whose low byte is the code.  The row stays in registers between the
// two steps, so x, r and g are read once and h and the codes written once: memory bound at
// 7 bytes per element (16-bit types with a residual) or 3 (token quantizer).
//
// Layout: NT threads per row (whole waves), NC chunks of VW consecutive elements per thread,
// VW = 8 (16-byte loads, 8-byte code stores) where the width and every pointer and stride
// allow it, else VW = 1 with lanes on consecutive elements.  The launch picks the widest
// thread count when there are fewer rows than compute units (latency), and otherwise fewer
// threads with more loads in flight each.
#include "../../include/pwq.h"
#include "pwq_internal.h"
#include "pwq_common.h"

namespace pwq {

namespace {

constexpr float TOK_TINY = 0x1p-120f;          // scales below this count as 0
constexpr double TOK_RINT = 0x1.8p52;          // x + this: nearest integer to x in the low bits
constexpr double TOK_SNAP = 0x1.8p22;          // x + this: x to a multiple of 2^-30
constexpr int64_t TOK_MAX_BLOCKS = 1 << 20;    // rows past this are taken by a loop in the kernel

struct TokArgs {
    const void* X;
    const void* R;                 // residual or NULL
    const void* G;                 // gain or NULL (all 1)
    const float* chan;             // channel scale or NULL
    void* H;                       // x + r in x's type, or NULL
    int8_t* Q;                     // codes or NULL
    float* S;
    int32_t* sums;
    void* Y;                       // normed rows or NULL
    int64_t ldx, ldr, ldh, ldq, ldy, T;
    double eps;
    int d, g_dtype, y_dtype;
};

// VW consecutive elements of a row, as they are stored
template <int XT, int VW>
struct Raw {
    static constexpr int N = VW == 1 ? 1 : (XT == 0 ? VW : VW / 2);
    uint32_t w[N];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        if constexpr (VW == 1) {
            w[0] = XT == 0 ? ((const uint32_t*)p)[i] : ((const uint16_t*)p)[i];
        } else {
            const uint4* v = (const uint4*)((const char*)p + i * (XT == 0 ? 4 : 2));
#pragma unroll
            for (int c = 0; c < N / 4; ++c) {
                const uint4 u = v[c];
                w[4 * c] = u.x; w[4 * c + 1] = u.y; w[4 * c + 2] = u.z; w[4 * c + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ void store(void* p, int64_t i) const {
        if constexpr (VW == 1) {
            if (XT == 0) ((uint32_t*)p)[i] = w[0];
            else ((uint16_t*)p)[i] = (uint16_t)w[0];
        } else {
            uint4* v = (uint4*)((char*)p + i * (XT == 0 ? 4 : 2));
#pragma unroll
            for (int c = 0; c < N / 4; ++c) v[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        }
    }
    __device__ __forceinline__ float get(int e) const {
        if (XT == 0) return __builtin_bit_cast(float, w[e]);
        const uint16_t b = (uint16_t)(VW == 1 ? w[0] : (e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu));
        return XT == 1 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int c = 0; c < N; ++c) w[c] = 0u;
    }
    // the sum a + b, rounded once to the type
    __device__ __forceinline__ void add(const Raw& a, const Raw& b) {
        if constexpr (XT == 0) {
#pragma unroll
            for (int e = 0; e < N; ++e) w[e] = __builtin_bit_cast(uint32_t, a.get(e) + b.get(e));
        } else {
            auto one = [&](int e) -> uint32_t {
                const float v = a.get(e) + b.get(e);
                return XT == 1 ? f32_to_f16_bits(v) : f32_to_bf16_bits(v);
            };
#pragma unroll
            for (int c = 0; c < N; ++c) w[c] = VW == 1 ? one(0) : (one(2 * c) | (one(2 * c + 1) << 16));
        }
    }
};

// VW gains from element i on (the type is the same for the whole launch); NULL: ones
template <int VW>
__device__ __forceinline__ void load_gain(float (&g)[VW], const void* G, int dtype, int64_t i) {
    if (!G) {
#pragma unroll
        for (int e = 0; e < VW; ++e) g[e] = 1.f;
    } else if (dtype == 0) {
        Raw<0, VW> r;
        r.load(G, i);
#pragma unroll
        for (int e = 0; e < VW; ++e) g[e] = r.get(e);
    } else if (dtype == 1) {
        Raw<1, VW> r;
        r.load(G, i);
#pragma unroll
        for (int e = 0; e < VW; ++e) g[e] = r.get(e);
    } else {
        Raw<2, VW> r;
        r.load(G, i);
#pragma unroll
        for (int e = 0; e < VW; ++e) g[e] = r.get(e);
    }
}

template <int VW>
__device__ __forceinline__ void store_y(void* Y, int dtype, int64_t i, const float (&y)[VW]) {
    auto put = [&](auto raw) {
        using R = decltype(raw);
#pragma unroll
        for (int c = 0; c < R::N; ++c) {
            if (dtype == 0) raw.w[c] = __builtin_bit_cast(uint32_t, y[c]);
            else {
                auto b = [&](int e) -> uint32_t { return dtype == 1 ? f32_to_f16_bits(y[e]) : f32_to_bf16_bits(y[e]); };
                raw.w[c] = VW == 1 ? b(0) : (b(2 * c) | (b(2 * c + 1) << 16));
            }
        }
        raw.store(Y, i);
    };
    if (dtype == 0) put(Raw<0, VW>{});
    else put(Raw<1, VW>{});
}

// low bytes of four float64 values that hold integers above 1.5 * 2^52
__device__ __forceinline__ uint32_t low_bytes(double a, double b, double c, double d) {
    const uint32_t x = (uint32_t)__double2loint(a), y = (uint32_t)__double2loint(b);
    const uint32_t z = (uint32_t)__double2loint(c), w = (uint32_t)__double2loint(d);
    const uint32_t lo = __builtin_amdgcn_perm(y, x, 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(w, z, 0x04000c0cu);
    return lo | hi;
}

struct SumMax {
    double sum, top;
};
__device__ __forceinline__ int lane_xor(int v, int o) { return __shfl_xor(v, o, WAVE); }
__device__ __forceinline__ SumMax lane_xor(SumMax v, int o) {
    return SumMax{__shfl_xor(v.sum, o, WAVE), __shfl_xor(v.top, o, WAVE)};
}

// over the NT threads of a row, the same value in all of them; slot: one entry per wave of the row
template <int NT, class T, class OP>
__device__ __forceinline__ T row_reduce(T v, T* slot, OP op) {
    constexpr int NW = NT / WAVE;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = op(v, lane_xor(v, o));
    if constexpr (NW > 1) {
        if ((threadIdx.x & 63) == 0) slot[(threadIdx.x % NT) / WAVE] = v;
        __syncthreads();
        v = slot[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) v = op(v, slot[w]);
    }
    return v;
}

template <int XT, int NT, int NC, int VW, bool NORM>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void tok_kernel(TokArgs a) {
    constexpr int RPB = NT < 256 ? 256 / NT : 1;          // rows per workgroup (one wave each)
    constexpr int NW = NT / WAVE;
    constexpr bool KEEP_G = NC * VW <= 16;                // gains loaded with the row, ahead of the reduction
    __shared__ SumMax red[2][NW];
    __shared__ int red_s[2][NW];
    const int tid = threadIdx.x % NT;
    const int d = a.d;
    int par = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / NT; row < a.T; row += (int64_t)gridDim.x * RPB, par ^= 1) {
        const char* xrow = (const char*)a.X + row * a.ldx * (XT == 0 ? 4 : 2);
        Raw<XT, VW> h[NC];
        float gain[KEEP_G && NORM ? NC : 1][VW];
        // every load is issued whether or not the chunk is inside the row (the address is
        // clamped and the value dropped), so that none waits behind a branch
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * NT + tid) * VW;
            h[c].load(xrow, col < d ? col : 0);
        }
        if constexpr (NORM) {
            if (a.R) {
                const char* rrow = (const char*)a.R + row * a.ldr * (XT == 0 ? 4 : 2);
                Raw<XT, VW> r[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int col = (c * NT + tid) * VW;
                    r[c].load(rrow, col < d ? col : 0);
                }
                if constexpr (KEEP_G) {
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int col = (c * NT + tid) * VW;
                        load_gain<VW>(gain[c], a.G, a.g_dtype, col < d ? col : 0);
                    }
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const Raw<XT, VW> x = h[c];
                    h[c].add(x, r[c]);
                    const int col = (c * NT + tid) * VW;
                    if (a.H && col < d) h[c].store((char*)a.H + row * a.ldh * (XT == 0 ? 4 : 2), col);
                }
            } else if constexpr (KEEP_G) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int col = (c * NT + tid) * VW;
                    load_gain<VW>(gain[c], a.G, a.g_dtype, col < d ? col : 0);
                }
            }
        }
        // y before the norm's factor: h g, or the token's own value (x / c)
        auto values = [&](int c, double (&p)[VW]) {
            const int col = (c * NT + tid) * VW;
            if constexpr (NORM) {
                float g[VW];
                if constexpr (KEEP_G) {
#pragma unroll
                    for (int e = 0; e < VW; ++e) g[e] = gain[c][e];
                } else {
                    load_gain<VW>(g, a.G, a.g_dtype, col < d ? col : 0);
                }
#pragma unroll
                for (int e = 0; e < VW; ++e) p[e] = (double)h[c].get(e) * (double)g[e];
            } else {
                Raw<0, VW> q;
                if (a.chan) q.load(a.chan, col < d ? col : 0);
#pragma unroll
                for (int e = 0; e < VW; ++e) p[e] = (double)(a.chan ? h[c].get(e) / q.get(e) : h[c].get(e));
            }
        };
        SumMax v{0.0, 0.0};
        double z = 0.0;                                   // NaN once a value is not finite
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if ((c * NT + tid) * VW < d) {
                double p[VW];
                values(c, p);
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    if constexpr (NORM) {
                        const double hd = (double)h[c].get(e);
                        v.sum = fma(hd, hd, v.sum);
                    }
                    v.top = fmax(v.top, fabs(p[e]));
                    z = fma(p[e], 0.0, z);
                }
            }
        }
        if (!(z == 0.0)) v.top = __builtin_inf();
        v = row_reduce<NT>(v, red[par], [](SumMax x, SumMax y) { return SumMax{x.sum + y.sum, fmax(x.top, y.top)}; });
        double rstd = 1.0;
        if constexpr (NORM) rstd = 1.0 / sqrt(v.sum / (double)d + a.eps);
        const bool bad = !(v.top < __builtin_inf()) || !(v.sum < __builtin_inf()) || !(rstd < __builtin_inf());
        float s = NORM ? (float)(v.top * rstd / 127.0) : (float)v.top / 127.0f;
        if (s < TOK_TINY) s = 0.f;
        if (bad) s = __builtin_nanf("");
        const bool live = s > 0.f;
        const double inv = live ? rstd / (double)s : 0.0;
        if (tid == 0 && a.S) a.S[row] = s;
        int sum = 0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * NT + tid) * VW;
            if (col >= d) continue;
            double p[VW];
            values(c, p);
            if (a.Q) {
                double q[VW];
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    // the norm's y / s is inexact by nature; the token quantizer's ties are exact:
                    // its quotients that are no tie are at least 2^-26 from one, so a step to
                    // the nearest multiple of 2^-30 makes ties exact and moves nothing across
                    q[e] = NORM ? fma(p[e], inv, TOK_RINT) : (fma(p[e], inv, TOK_SNAP) - TOK_SNAP) + TOK_RINT;
                }
                if constexpr (VW == 1) {
                    const int code = live ? (int)(int8_t)__double2loint(q[0]) : 0;
                    a.Q[row * a.ldq + col] = (int8_t)code;
                    sum += code;
                } else {
                    uint32_t w[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        w[k] = live ? low_bytes(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]) : 0u;
                        sum = __builtin_amdgcn_sdot4((int)w[k], 0x01010101, sum, false);
                    }
                    *(uint2*)(a.Q + row * a.ldq + col) = make_uint2(w[0], w[1]);
                }
            }
            if constexpr (NORM) {
                if (a.Y) {
                    float y[VW];
#pragma unroll
                    for (int e = 0; e < VW; ++e) y[e] = (float)(p[e] * rstd);
                    store_y<VW>((char*)a.Y + row * a.ldy * (a.y_dtype == 0 ? 4 : 2), a.y_dtype, col, y);
                }
            }
        }
        if (a.sums) {
            sum = row_reduce<NT>(sum, red_s[par], [](int x, int y) { return x + y; });
            if (tid == 0) a.sums[row] = sum;
        }
    }
}

template <int XT, int NT, int NC, int VW, bool NORM>
hipError_t tok_go(const TokArgs& a, hipStream_t s) {
    constexpr int RPB = NT < 256 ? 256 / NT : 1;
    const int64_t blocks = cdiv(a.T, RPB);
    hipLaunchKernelGGL((tok_kernel<XT, NT, NC, VW, NORM>), dim3((unsigned)(blocks < TOK_MAX_BLOCKS ? blocks : TOK_MAX_BLOCKS)),
                       dim3(NT < 256 ? 256 : NT), 0, s, a);
    return hipGetLastError();
}

template <int XT, bool NORM>
hipError_t tok_pick(const TokArgs& a, bool vec, hipStream_t s) {
    const int d = a.d;
    const bool few = a.T < 256;                           // fewer rows than compute units
    if (vec) {
        if (d <= 512) return tok_go<XT, 64, 1, 8, NORM>(a, s);
        if (d <= 1024) return tok_go<XT, 64, 2, 8, NORM>(a, s);
        if (d <= 2048 && few) return tok_go<XT, 256, 1, 8, NORM>(a, s);
        if (d <= 2048) return tok_go<XT, 64, 4, 8, NORM>(a, s);
        if (d <= 8192 && few) return tok_go<XT, 1024, 1, 8, NORM>(a, s);
        if (d <= 4096) return tok_go<XT, 256, 2, 8, NORM>(a, s);
        if (d <= 8192) return tok_go<XT, 256, 4, 8, NORM>(a, s);
        if (d <= 16384) return tok_go<XT, 1024, 2, 8, NORM>(a, s);
        if (d <= 32768) return tok_go<XT, 1024, 4, 8, NORM>(a, s);
        return tok_go<XT, 1024, 8, 8, NORM>(a, s);
    }
    if (d <= 512) return tok_go<XT, 64, 8, 1, NORM>(a, s);
    if (d <= 2048) return tok_go<XT, 256, 8, 1, NORM>(a, s);
    if (d <= 8192) return tok_go<XT, 1024, 8, 1, NORM>(a, s);
    if (d <= 16384) return tok_go<XT, 1024, 16, 1, NORM>(a, s);
    return tok_go<XT, 1024, 64, 1, NORM>(a, s);
}

// 16-byte loads and stores of 8 elements (8-byte ones for codes) at every multiple of 8
bool rows16(const void* p, int64_t ld, int dtype) {
    if (!p) return true;
    return aligned(p, 16) && ld * (dtype == 0 ? 4 : 2) % 16 == 0;
}

}  // namespace

hipError_t tok_quant_launch(const void* X, int x_dtype, int64_t T, int64_t d, int64_t ldx, const float* chan, int8_t* Q,
                            int64_t ldq, float* S, int32_t* sums, hipStream_t s) {
    TokArgs a{};
    a.X = X; a.ldx = ldx; a.T = T; a.d = (int)d; a.chan = chan;
    a.Q = Q; a.ldq = ldq; a.S = S; a.sums = sums;
    const bool vec = d % 8 == 0 && rows16(X, ldx, x_dtype) && rows16(chan, 4, 0) && aligned(Q, 8) && ldq % 8 == 0;
    if (x_dtype == 0) return tok_pick<0, false>(a, vec, s);
    if (x_dtype == 1) return tok_pick<1, false>(a, vec, s);
    return tok_pick<2, false>(a, vec, s);
}

hipError_t rms_norm_launch(const void* X, int x_dtype, int64_t T, int64_t d, int64_t ldx, const void* R, int64_t ldr,
                           const void* G, int g_dtype, double eps, void* H, int64_t ldh, int8_t* Q, int64_t ldq, float* S,
                           int32_t* sums, void* Y, int y_dtype, int64_t ldy, hipStream_t s) {
    TokArgs a{};
    a.X = X; a.ldx = ldx; a.T = T; a.d = (int)d; a.R = R; a.ldr = ldr; a.G = G; a.g_dtype = g_dtype; a.eps = eps;
    a.H = H; a.ldh = ldh; a.Q = Q; a.ldq = ldq; a.S = S; a.sums = sums; a.Y = Y; a.y_dtype = y_dtype; a.ldy = ldy;
    const bool vec = d % 8 == 0 && rows16(X, ldx, x_dtype) && rows16(R, ldr, x_dtype) && rows16(H, ldh, x_dtype) &&
                     rows16(G, 8, g_dtype) && rows16(Y, ldy, y_dtype) && (!Q || (aligned(Q, 8) && ldq % 8 == 0));
    if (x_dtype == 0) return tok_pick<0, true>(a, vec, s);
    if (x_dtype == 1) return tok_pick<1, true>(a, vec, s);
    return tok_pick<2, true>(a, vec, s);
}

}  // namespace pwq
