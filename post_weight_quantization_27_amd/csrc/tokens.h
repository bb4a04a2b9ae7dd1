// 8-bit codes of activations, one symmetric scale per token, alone (pwq_quantize_tokens) and
// fused with the root-mean-square norm and the residual's addition (pwq_rms_norm_quantize):
// the X operand of the int8 product (pwq_quantized_matmul_int8).
//
// Per row of values y:
//   s = float32(max |y| / 127); s below 2^-120 counts as 0, a value that is not finite makes s NaN;
//   code = nearest integer to y / s, ties to even (s = 0 or NaN: code 0).
// Token quantizer: y = x, or the float32 quotient x / c with a scale c per channel.
// Norm: h = x + r rounded once to x's type, y = h g / sqrt(mean(h^2) + eps).  Since
// max |y| = rstd max |h g|, the sum of squares and the largest |h g| come out of ONE pass over
// the row and one reduction; the codes are then nearest(h g (rstd / s)).
//
// A code next to a border between two levels has to come out as the 64-bit definition says,
// whatever the order of the sum, so the sum of squares, rstd and the quotient are float64 (whose
// fma runs at the float32 rate on this chip).  The products h g of 16-bit values have at most 22
// significant bits and are formed in float32, exactly while the largest is in [2^-60, inf):
// smaller ones that float32 cannot hold are below 2^-66 of the largest and get code 0 either way.
// Rows outside that range (zeros, overflow, NaN) and float32 inputs go through float64 products.
// The nearest integer is one fma with 1.5 * 2^52 added, whose low byte is the code.
//
// The row stays in registers between the two steps, so x, r and g are read once and h and the
// codes written once: memory bound at 7 bytes per element (16-bit types with a residual) or 3
// (token quantizer).
//
// Layout: NT threads per row (whole waves), NC chunks of 8 consecutive elements per thread: few
// threads with several chunks, so that a compute unit has several rows in flight and one's loads
// run beside another's stores.  Rows too long for the registers are read again for the second
// step.  Measured (kernel trace, operands cold): norm of 8192 x 8192 bf16 with a residual 96 us (4.9
// TB/s, as a copy of as many bytes), in float32 183 (4.8), with a float32 gain 102, rows that start
// at any byte 137; token quantizer of 4096 x 28672 bf16 81 us (4.4 TB/s), float32 112 (5.2), with a
// channel scale 122 (the scales, twice X's bytes, are loaded from L2 and divided by for every row);
// one row of 8192 4.8 us, an empty launch 2.2.
#pragma once

#include "../../include/pwq.h"
#include "pwq_internal.h"
#include "pwq_common.h"

namespace pwq {

namespace {

constexpr float TOK_TINY = 0x1p-120f;          // scales below this count as 0
constexpr double TOK_RINT = 0x1.8p52;          // x + this: nearest integer to x in the low bits
constexpr double TOK_SNAP = 0x1.8p22;          // x + this: x to a multiple of 2^-30
constexpr float TOK_LOW = 0x1p-60f;            // float32 products of 16-bit values are used from here on
constexpr int64_t TOK_MAX_BLOCKS = 1 << 20;    // rows past this are taken by a loop in the kernel

// y = x, y = x / c; the norm with float32 products of 16-bit values, with float64 products
enum { TOK_PLAIN, TOK_CHAN, TOK_NORM16, TOK_NORM64 };

// Rows: 16-byte loads and stores of eight elements at multiples of their size (a width that is a
// multiple of 8), at any address, and rows shorter than eight elements
enum { ROWS_VEC, ROWS_ANY, ROWS_SHORT };

struct TokArgs {
    const void* X;
    const void* R;                 // residual or NULL
    const void* G;                 // gain or NULL (all 1)
    const float* chan;             // channel scale
    void* H;                       // x + r in x's type, or NULL
    int8_t* Q;                     // codes or NULL
    float* S;
    int32_t* sums;
    void* Y;                       // normed rows or NULL
    int64_t ldx, ldr, ldh, ldq, ldy, T;
    double eps;
    int d, g_dtype, y_dtype;
};

template <int XT>
__device__ __forceinline__ float from_bits16(uint32_t b) {
    return XT == 1 ? f16_bits_to_f32((uint16_t)b) : bf16_bits_to_f32((uint16_t)b);
}

// Eight consecutive elements of a row, as they are stored
template <int XT>
struct Raw {
    static constexpr int N = XT == 0 ? 8 : 4;
    static constexpr int SIZE = XT == 0 ? 4 : 2;
    uint32_t w[N];
    // Elements col .. col + 7 of a row of d, zeros past its end, in two parts: all of a row's chunks
    // are fetched before the first is settled, which waits for it.  ROWS_ANY: the chunk that
    // passes the end is fetched from d - 8 on and moved down.  No load stands behind a branch.  A
    // chunk wholly past the end is fetched from somewhere in the row and not used.
    template <int AL>
    __device__ __forceinline__ void fetch(const void* row, int col, int d) {
        if constexpr (AL == ROWS_VEC) {
            const uint4* v = (const uint4*)((const char*)row + (int64_t)(col < d ? col : 0) * SIZE);
#pragma unroll
            for (int c = 0; c < N / 4; ++c) {
                const uint4 u = v[c];
                w[4 * c] = u.x; w[4 * c + 1] = u.y; w[4 * c + 2] = u.z; w[4 * c + 3] = u.w;
            }
        } else if constexpr (AL == ROWS_ANY) {
            __builtin_memcpy(w, (const char*)row + (int64_t)(col < d - 8 ? col : d - 8) * SIZE, 8 * SIZE);
        } else {
            zero();
            if (col == 0) {
                for (int e = 0; e < d; ++e) {
                    if (XT == 0) set(e, ((const uint32_t*)row)[e]);
                    else set(e, ((const uint16_t*)row)[e]);
                }
            }
        }
    }
    template <int AL>
    __device__ __forceinline__ void settle(int col, int d) {
        if (AL == ROWS_ANY && col > d - 8 && col < d) down(col - (d - 8));
    }
    template <int AL>
    __device__ __forceinline__ void load(const void* row, int col, int d) {
        fetch<AL>(row, col, d);
        settle<AL>(col, d);
    }
    // Elements col .. min(col + 8, d) - 1 into the row
    template <int AL>
    __device__ __forceinline__ void store(void* row, int col, int d) const {
        char* p = (char*)row + (int64_t)col * SIZE;
        if constexpr (AL == ROWS_VEC) {
#pragma unroll
            for (int c = 0; c < N / 4; ++c) ((uint4*)p)[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        } else if (col + 8 <= d) {
            __builtin_memcpy(p, w, 8 * SIZE);
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e) {
                if (col + e < d) {
                    if (XT == 0) ((uint32_t*)p)[e] = w[e % N];
                    else ((uint16_t*)p)[e] = (uint16_t)(e & 1 ? w[e / 2] >> 16 : w[e / 2]);
                }
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int c = 0; c < N; ++c) w[c] = 0u;
    }
    __device__ __forceinline__ void set(int e, uint32_t bits) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i != e) continue;
            if (XT == 0) w[i % N] = bits;
            else w[i / 2] |= bits << (16 * (i & 1));
        }
    }
    // element e <- element e + by, zeros from the end
    __device__ __forceinline__ void down(int by) {
        if constexpr (XT != 0) {
            if (by & 1) {
#pragma unroll
                for (int c = 0; c < N; ++c) w[c] = (w[c] >> 16) | (c + 1 < N ? w[(c + 1) % N] << 16 : 0u);
            }
            by >>= 1;
        }
#pragma unroll
        for (int b = 1; b < N; b *= 2) {
            if (by & b) {
#pragma unroll
                for (int c = 0; c < N; ++c) w[c] = c + b < N ? w[(c + b) % N] : 0u;
            }
        }
    }
    __device__ __forceinline__ float get(int e) const {
        if (XT == 0) return __builtin_bit_cast(float, w[e % N]);
        return from_bits16<XT>(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu);
    }
    // the sum a + b, rounded once to the type
    __device__ __forceinline__ void add(const Raw& a, const Raw& b) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
            if constexpr (XT == 0) {
                w[c] = __builtin_bit_cast(uint32_t, a.get(c) + b.get(c));
            } else {
                const float lo = a.get(2 * c) + b.get(2 * c), hi = a.get(2 * c + 1) + b.get(2 * c + 1);
                w[c] = XT == 1 ? (uint32_t)f32_to_f16_bits(lo) | ((uint32_t)f32_to_f16_bits(hi) << 16)
                               : (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
            }
        }
    }
};

// y of eight elements, rounded to y_dtype
template <int AL>
__device__ __forceinline__ void store_y(const TokArgs& a, int64_t row, int col, const float (&y)[8]) {
    char* p = (char*)a.Y + row * a.ldy * (a.y_dtype == 0 ? 4 : 2);
    if (a.y_dtype == 0) {
        Raw<0> r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.w[e] = __builtin_bit_cast(uint32_t, y[e]);
        r.template store<AL>(p, col, a.d);
    } else {
        Raw<1> r;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float lo = y[2 * c], hi = y[2 * c + 1];
            r.w[c] = a.y_dtype == 1 ? (uint32_t)f32_to_f16_bits(lo) | ((uint32_t)f32_to_f16_bits(hi) << 16)
                                    : (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
        }
        r.template store<AL>(p, col, a.d);
    }
}

// eight codes, from float64 values whose low byte each is, into the row; returns their sum
template <int AL>
__device__ __forceinline__ int store_codes(int8_t* q, int col, int d, const double (&v)[8], bool live) {
    uint32_t w[2];
    int sum = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t b0 = (uint32_t)__double2loint(v[4 * k]), b1 = (uint32_t)__double2loint(v[4 * k + 1]);
        const uint32_t b2 = (uint32_t)__double2loint(v[4 * k + 2]), b3 = (uint32_t)__double2loint(v[4 * k + 3]);
        w[k] = __builtin_amdgcn_perm(b1, b0, 0x0c0c0400u) | __builtin_amdgcn_perm(b3, b2, 0x04000c0cu);
        if (!live) w[k] = 0u;
        // past the end of a row the values are 0, and so are these codes
        sum = __builtin_amdgcn_sdot4((int)w[k], 0x01010101, sum, false);
    }
    if constexpr (AL == ROWS_VEC) {
        *(uint2*)(q + col) = make_uint2(w[0], w[1]);
    } else if (col + 8 <= d) {
        __builtin_memcpy(q + col, w, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (col + e < d) q[col + e] = (int8_t)(w[e / 4] >> (8 * (e & 3)));
    }
    return sum;
}

// The larger of a and b >= 0, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

struct SumMax {
    double sum, top;
};
struct SumMaxF {
    double sum;
    float top;
};
__device__ __forceinline__ int lane_xor(int v, int o) { return __shfl_xor(v, o, WAVE); }
__device__ __forceinline__ float lane_xor(float v, int o) { return __shfl_xor(v, o, WAVE); }
__device__ __forceinline__ SumMax lane_xor(SumMax v, int o) {
    return SumMax{__shfl_xor(v.sum, o, WAVE), __shfl_xor(v.top, o, WAVE)};
}
__device__ __forceinline__ SumMaxF lane_xor(SumMaxF v, int o) {
    return SumMaxF{__shfl_xor(v.sum, o, WAVE), __shfl_xor(v.top, o, WAVE)};
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

// The scale of a row whose largest |y| is top (not finite: NaN), and whether its codes are other than 0
struct Scale {
    float s;
    bool live;
};
__device__ __forceinline__ Scale tok_scale(float s, bool finite) {
    if (s < TOK_TINY) s = 0.f;
    if (!finite) s = __builtin_nanf("");
    return Scale{s, s > 0.f};
}

// LDS of a workgroup; two of each, used by rows in turn, so that one barrier per reduction is enough
template <int NW>
struct TokLds {
    SumMax sm[2][NW];
    SumMaxF smf[2][NW];
    float top[2][NW];
    int bits[2][NW], sum[2][NW];
};

// One row of the norm in float64 products, read from memory in each of its two steps: rows that
// the float32 products do not cover, and rows too long for the registers.  h_done: h has been
// written to a.H already (by the same threads, the same elements), and x may be gone with it.
template <int XT, int NT, int AL>
__device__ void norm_row_mem(const TokArgs& a, int64_t row, int par, TokLds<NT / WAVE>& lds, bool h_done) {
    const int tid = threadIdx.x % NT;
    constexpr int SIZE = Raw<XT>::SIZE;
    const char* xrow = (const char*)a.X + row * a.ldx * SIZE;
    const char* rrow = a.R ? (const char*)a.R + row * a.ldr * SIZE : nullptr;
    char* hrow = a.H ? (char*)a.H + row * a.ldh * SIZE : nullptr;
    auto read = [&](int col, Raw<XT>& h, float (&g)[8], bool from_h) {
        if (from_h) {
            h.template load<AL>(hrow, col, a.d);
        } else {
            h.template load<AL>(xrow, col, a.d);
            if (rrow) {
                Raw<XT> r;
                r.template load<AL>(rrow, col, a.d);
                h.add(h, r);
            }
        }
        auto gains = [&](auto raw) {
            raw.template load<AL>(a.G, col, a.d);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = raw.get(e);
        };
        if (!a.G) {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = 1.f;
        } else if (a.g_dtype == 0) {
            gains(Raw<0>{});
        } else if (a.g_dtype == 1) {
            gains(Raw<1>{});
        } else {
            gains(Raw<2>{});
        }
    };
    SumMax v{0.0, 0.0};
    double z = 0.0;                                       // NaN once a product is not finite
    for (int col = tid * 8; col < a.d; col += NT * 8) {
        Raw<XT> h;
        float g[8];
        read(col, h, g, h_done && hrow);
        if (!h_done && hrow) h.template store<AL>(hrow, col, a.d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double hd = (double)h.get(e), p = hd * (double)g[e];
            v.sum = fma(hd, hd, v.sum);
            v.top = fmax(v.top, fabs(p));
            z = fma(p, 0.0, z);
        }
    }
    if (!(z == 0.0)) v.top = __builtin_inf();
    v = row_reduce<NT>(v, lds.sm[par], [](SumMax x, SumMax y) { return SumMax{x.sum + y.sum, fmax(x.top, y.top)}; });
    const double rstd = 1.0 / sqrt(v.sum / (double)a.d + a.eps);
    const bool finite = v.top < __builtin_inf() && v.sum < __builtin_inf() && rstd < __builtin_inf();
    const Scale s = tok_scale((float)(v.top * rstd / 127.0), finite);
    const double inv = s.live ? rstd / (double)s.s : 0.0;
    if (tid == 0 && a.S) a.S[row] = s.s;
    int sum = 0;
    for (int col = tid * 8; col < a.d; col += NT * 8) {
        Raw<XT> h;
        float g[8], y[8];
        double q[8];
        read(col, h, g, hrow != nullptr);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double p = (double)h.get(e) * (double)g[e];
            q[e] = fma(p, inv, TOK_RINT);
            y[e] = (float)(p * rstd);
        }
        if (a.Q) sum += store_codes<AL>(a.Q + row * a.ldq, col, a.d, q, s.live);
        if (a.Y) store_y<AL>(a, row, col, y);
    }
    if (a.sums) {
        sum = row_reduce<NT>(sum, lds.sum[par], [](int x, int y) { return x + y; });
        if (tid == 0) a.sums[row] = sum;
    }
}

// One row of the token quantizer, read from memory in each of its two steps: rows too long for the
// registers.
template <int XT, int NT, int AL>
__device__ void tok_row_mem(const TokArgs& a, int64_t row, int par, TokLds<NT / WAVE>& lds) {
    const int tid = threadIdx.x % NT;
    const char* xrow = (const char*)a.X + row * a.ldx * Raw<XT>::SIZE;
    auto read = [&](int col, float (&y)[8]) {
        Raw<XT> x;
        x.template load<AL>(xrow, col, a.d);
        Raw<0> c;
        if (a.chan) c.template load<AL>(a.chan, col, a.d);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = !a.chan || (AL != ROWS_VEC && col + e >= a.d) ? x.get(e) : x.get(e) / c.get(e);
    };
    float top = 0.f;
    for (int col = tid * 8; col < a.d; col += NT * 8) {
        float y[8];
        read(col, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(y[e]));
    }
    top = row_reduce<NT>(top, lds.top[par], [](float x, float y) { return max_nan(x, y); });
    const Scale s = tok_scale(top / 127.0f, top < __builtin_inff());
    const double inv = s.live ? 1.0 / (double)s.s : 0.0;
    if (tid == 0) a.S[row] = s.s;
    int sum = 0;
    for (int col = tid * 8; col < a.d; col += NT * 8) {
        float y[8];
        double q[8];
        read(col, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = (fma((double)y[e], inv, TOK_SNAP) - TOK_SNAP) + TOK_RINT;
        sum += store_codes<AL>(a.Q + row * a.ldq, col, a.d, q, s.live);
    }
    if (a.sums) {
        sum = row_reduce<NT>(sum, lds.sum[par], [](int x, int y) { return x + y; });
        if (tid == 0) a.sums[row] = sum;
    }
}

template <int XT, int NT, bool NORM, int AL>
__global__ __launch_bounds__(NT) void tok_mem_kernel(TokArgs a) {
    __shared__ TokLds<NT / WAVE> lds;
    int par = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, par ^= 1) {
        if constexpr (NORM) norm_row_mem<XT, NT, AL>(a, row, par, lds, false);
        else tok_row_mem<XT, NT, AL>(a, row, par, lds);
    }
}

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

template <int XT, int NT, int NC, int MODE, int AL>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void tok_kernel(TokArgs a) {
    constexpr int RPB = NT < 256 ? 256 / NT : 1;          // rows per workgroup (one wave each)
    constexpr bool NORM = MODE >= TOK_NORM16;
    constexpr int SIZE = Raw<XT>::SIZE;
    __shared__ TokLds<NT / WAVE> lds;
    const int tid = threadIdx.x % NT;
    const int d = a.d;
    auto col_of = [&](int c) { return (c * NT + tid) * 8; };
    int par = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / NT; row < a.T; row += (int64_t)gridDim.x * RPB, par ^= 1) {
        // every load of the row is issued before the first value is used
        const char* xrow = (const char*)a.X + row * a.ldx * SIZE;
        Raw<XT> h[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) h[c].template fetch<AL>(xrow, col_of(c), d);
        if constexpr (NORM) {
            if (a.R) {
                const char* rrow = (const char*)a.R + row * a.ldr * SIZE;
                Raw<XT> r[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c) r[c].template fetch<AL>(rrow, col_of(c), d);
#pragma unroll
                for (int c = 0; c < NC; ++c) h[c].add(h[c], r[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) h[c].template settle<AL>(col_of(c), d);
        double rstd = 1.0;
        Scale s;
        double inv;
        float v[MODE == TOK_CHAN || MODE == TOK_NORM16 ? NC : 1][8];   // x / c, or h g
        float g[MODE == TOK_NORM64 ? NC : 1][8];

        if constexpr (MODE == TOK_PLAIN && XT != 0) {
            // 16-bit magnitudes order like their bits, two at a time
            u16x2 top = {0, 0};
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (col_of(c) >= d) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, h[c].w[k % Raw<XT>::N] & 0x7fff7fffu));
            }
            int bits = top[0] > top[1] ? top[0] : top[1];
            bits = row_reduce<NT>(bits, lds.bits[par], [](int x, int y) { return x > y ? x : y; });
            s = tok_scale(from_bits16<XT>((uint32_t)bits) / 127.0f, bits < (XT == 1 ? 0x7c00 : 0x7f80));
        } else if constexpr (!NORM) {
            if constexpr (MODE == TOK_CHAN) {
                Raw<0> cs[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c) cs[c].template fetch<AL>(a.chan, col_of(c), d);
#pragma unroll
                for (int c = 0; c < NC; ++c) cs[c].template settle<AL>(col_of(c), d);
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[c][e] = AL == ROWS_VEC || col_of(c) + e < d ? h[c].get(e) / cs[c].get(e) : 0.f;
            }
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (col_of(c) >= d) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(MODE == TOK_CHAN ? v[c % NC][e] : h[c].get(e)));
            }
            top = row_reduce<NT>(top, lds.top[par], [](float x, float y) { return max_nan(x, y); });
            s = tok_scale(top / 127.0f, top < __builtin_inff());
        } else {
            SumMaxF m{0.0, 0.f};
            SumMax m64{0.0, 0.0};
            double z = 0.0;
            if constexpr (MODE == TOK_NORM16) {
                auto products = [&](auto raw) {
                    using G = decltype(raw);
                    G gr[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c) gr[c].template fetch<AL>(a.G, col_of(c), d);
#pragma unroll
                    for (int c = 0; c < NC; ++c) gr[c].template settle<AL>(col_of(c), d);
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[c][e] = h[c].get(e) * gr[c].get(e);
                    if (a.Y) {
                        // y itself is wanted too: a product that float32 cannot hold exactly sends the
                        // row to the float64 products (22 bits from 2^-126 on)
                        bool low = false;
#pragma unroll
                        for (int c = 0; c < NC; ++c)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                low |= fabsf(v[c][e]) < 0x1p-100f && h[c].get(e) != 0.f && gr[c].get(e) != 0.f;
                        if (low) m.top = __builtin_inff();
                    }
                };
                if (!a.G) {
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[c][e] = h[c].get(e);
                } else if (a.g_dtype == 1) {
                    products(Raw<1>{});
                } else {
                    products(Raw<2>{});
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if (col_of(c) >= d) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const double hd = (double)h[c].get(e);
                        m.sum = fma(hd, hd, m.sum);
                        m.top = max_nan(m.top, fabsf(v[c][e]));
                    }
                }
            } else {
                auto gains = [&](auto raw) {
                    using G = decltype(raw);
                    G gr[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c) gr[c].template fetch<AL>(a.G, col_of(c), d);
#pragma unroll
                    for (int c = 0; c < NC; ++c) gr[c].template settle<AL>(col_of(c), d);
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[c][e] = gr[c].get(e);
                };
                if (!a.G) {
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[c][e] = 1.f;
                } else if (a.g_dtype == 0) {
                    gains(Raw<0>{});
                } else if (a.g_dtype == 1) {
                    gains(Raw<1>{});
                } else {
                    gains(Raw<2>{});
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if (col_of(c) >= d) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const double hd = (double)h[c].get(e), p = hd * (double)g[c][e];
                        m64.sum = fma(hd, hd, m64.sum);
                        m64.top = fmax(m64.top, fabs(p));
                        z = fma(p, 0.0, z);
                    }
                }
            }
            if (a.H) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (col_of(c) < d) h[c].template store<AL>((char*)a.H + row * a.ldh * SIZE, col_of(c), d);
            }
            bool finite;
            if constexpr (MODE == TOK_NORM16) {
                m = row_reduce<NT>(m, lds.smf[par], [](SumMaxF x, SumMaxF y) { return SumMaxF{x.sum + y.sum, max_nan(x.top, y.top)}; });
                if (!(m.top >= TOK_LOW && m.top < __builtin_inff())) {   // the same for every thread of the row
                    norm_row_mem<XT, NT, AL>(a, row, par, lds, a.H != nullptr);
                    continue;
                }
                m64 = SumMax{m.sum, (double)m.top};
            } else {
                if (!(z == 0.0)) m64.top = __builtin_inf();
                m64 = row_reduce<NT>(m64, lds.sm[par], [](SumMax x, SumMax y) { return SumMax{x.sum + y.sum, fmax(x.top, y.top)}; });
            }
            rstd = 1.0 / sqrt(m64.sum / (double)d + a.eps);
            finite = m64.top < __builtin_inf() && m64.sum < __builtin_inf() && rstd < __builtin_inf();
            s = tok_scale((float)(m64.top * rstd / 127.0), finite);
        }
        inv = s.live ? rstd / (double)s.s : 0.0;
        if (tid == 0 && a.S) a.S[row] = s.s;

        int sum = 0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = col_of(c);
            if (col >= d) continue;
            double p[8], q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (MODE == TOK_NORM64) p[e] = (double)h[c].get(e) * (double)g[c][e];
                else if constexpr (MODE == TOK_PLAIN) p[e] = (double)h[c].get(e);
                else p[e] = (double)v[c % NC][e];
                // The norm's y / s is inexact by nature.  The token quantizer's quotients that are no
                // tie are at least 2^-26 from one, so a step to the nearest multiple of 2^-30 makes
                // ties exact and moves nothing across them.
                q[e] = NORM ? fma(p[e], inv, TOK_RINT) : (fma(p[e], inv, TOK_SNAP) - TOK_SNAP) + TOK_RINT;
            }
            if (!NORM || a.Q) sum += store_codes<AL>(a.Q + row * a.ldq, col, d, q, s.live);
            if constexpr (NORM) {
                if (a.Y) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = (float)(p[e] * rstd);
                    store_y<AL>(a, row, col, y);
                }
            }
        }
        if (a.sums) {
            sum = row_reduce<NT>(sum, lds.sum[par], [](int x, int y) { return x + y; });
            if (tid == 0) a.sums[row] = sum;
        }
    }
}

template <int XT, int NT, int NC, int MODE, int AL>
hipError_t tok_go(const TokArgs& a, hipStream_t s) {
    constexpr int RPB = NT < 256 ? 256 / NT : 1;
    const int64_t blocks = cdiv(a.T, RPB);
    hipLaunchKernelGGL((tok_kernel<XT, NT, NC, MODE, AL>),
                       dim3((unsigned)(blocks < TOK_MAX_BLOCKS ? blocks : TOK_MAX_BLOCKS)), dim3(NT < 256 ? 256 : NT), 0, s, a);
    return hipGetLastError();
}

// Rows read from memory in both steps
template <int XT, int NT, int MODE, int AL>
hipError_t tok_go_mem(const TokArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((tok_mem_kernel<XT, NT, (MODE >= TOK_NORM16), AL>),
                       dim3((unsigned)(a.T < TOK_MAX_BLOCKS ? a.T : TOK_MAX_BLOCKS)), dim3(NT), 0, s, a);
    return hipGetLastError();
}

template <int XT, int MODE, int AL>
hipError_t tok_pick(const TokArgs& a, hipStream_t s) {
    const int64_t d = cdiv(a.d, 8) * 8;
    // One wave per row while it holds the row (16384 x 768 float16: 10.6 against 20.4 us with 256
    // threads; the same at 1 row), then 256 threads (8192 x 8192 norm: 92 us, with 512 threads of
    // 2 chunks 99, 1024 of one 160; 1 row: 4.3 / 4.2 / 4.9) with no more chunks than needed (norm of
    // 8192 x 5120: 59 us with 3, 63 with 4), then 512 (4096 x 28672: 70 us, with 1024 of 4 chunks
    // 75; 16 rows: 4.9 either way).
    if (d <= 1024) return tok_go<XT, 64, 2, MODE, AL>(a, s);
    if (d <= 2048) return tok_go<XT, 256, 1, MODE, AL>(a, s);
    if (d <= 4096) return tok_go<XT, 256, 2, MODE, AL>(a, s);
    if (d <= 6144) return tok_go<XT, 256, 3, MODE, AL>(a, s);
    if (d <= 8192) return tok_go<XT, 256, 4, MODE, AL>(a, s);
    // Longer rows: as far as the registers hold them (the norm holds x, r and g at once, the float64
    // products the gains beside h, unaligned rows the shifted chunks), since a row read twice takes
    // longer: token quantizer 81 us at 4096 x 28672, 129 at 28671, which is read twice; norm with a
    // residual 177 at 28672 against 250 at 32768.  The norm of 16-bit rows in seven chunks is the one
    // that spills (8 registers of a lane: 67 MB more written over 4096 rows, 19 % at 28672 wide) and is
    // still ahead.  Rows between the steps pay for the chunks they leave empty: norm of 4096 rows
    // of 16384 / 18944 / 20480 / 24576 / 28672: 103 / 132 / 137 / 160 / 177 us.
    if constexpr (AL == ROWS_VEC || MODE != TOK_NORM64) {
        if (d <= 16384) return tok_go<XT, 512, 4, MODE, AL>(a, s);
    }
    if constexpr (AL == ROWS_VEC && MODE != TOK_NORM64) {
        if (d <= 28672) return tok_go<XT, 512, 7, MODE, AL>(a, s);
    }
    if constexpr (AL == ROWS_VEC && MODE < TOK_NORM16) {
        if (d <= 32768) return tok_go<XT, 512, 8, MODE, AL>(a, s);
    }
    return tok_go_mem<XT, 1024, MODE, AL>(a, s);
}

template <int XT, int MODE>
hipError_t tok_rows(const TokArgs& a, bool vec, hipStream_t s) {
    if (vec) return tok_pick<XT, MODE, ROWS_VEC>(a, s);
    if (a.d >= 8) return tok_pick<XT, MODE, ROWS_ANY>(a, s);
    return tok_go_mem<XT, 64, MODE, ROWS_SHORT>(a, s);
}

template <int MODE>
hipError_t tok_type(const TokArgs& a, int x_dtype, bool vec, hipStream_t s) {
    if constexpr (MODE != TOK_NORM16) {
        if (x_dtype == 0) return tok_rows<0, MODE>(a, vec, s);
    }
    return x_dtype == 1 ? tok_rows<1, MODE>(a, vec, s) : tok_rows<2, MODE>(a, vec, s);
}

// 16-byte loads and stores of 8 elements (8-byte ones for codes) at every multiple of 8
inline bool rows16(const void* p, int64_t ld, int dtype) {
    if (!p) return true;
    return aligned(p, 16) && ld * (dtype == 0 ? 4 : 2) % 16 == 0;
}

}  // namespace

}  // namespace pwq
