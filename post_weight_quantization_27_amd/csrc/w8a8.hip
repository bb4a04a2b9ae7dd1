// Product of 8-bit codes with 8-bit codes, exact sums, one scale per token and per output row:
//
//   Y[t, o] = sx[t] sw[o] sum_k X[t, k] (C[o, k] - z[o])
//
// X: int8 codes of activations (pwq_quantize_tokens, pwq_rms_norm_quantize); C: a layer's codes
// (RTN or GPTQ at up to 8 bits, one scale per row), int8 with z = 0, or the unsigned codes of
// the zero-point form with z per row.  There the sum is taken over the signed bytes C - 128
// (the byte with its top bit flipped) and (128 - z[o]) sum_k X[t, k] is added: the token sums
// come with X's codes.  All sums are int32 and exact (d_in <= 65535 keeps them below 2^31), so
// neither the order nor the split of k changes a bit; the float result is rounded by the
// conversion of the sum, the two scales and the store.
//
// The multiply runs on v_mfma_i32_32x32x32_i8 with X as the row operand (tokens) and C as the
// column operand (outputs): a lane holds 16 consecutive k of one row of each, in any order of k
// as long as both operands agree.
#include "../../include/pwq.h"
#include "pwq_internal.h"
#include "pwq_common.h"

namespace pwq {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int W8_SPLIT_MIN_K = 512;        // least k of a split

struct W8Args {
    const int8_t* X;
    const float* sx;
    const int32_t* sums;           // token sums (zero-point form) or NULL
    const uint8_t* C;              // d_out x d_in, dense
    const uint16_t* sw;            // float16 bits
    const uint16_t* zeros;         // zero-point form or NULL
    void* Y;
    int32_t* part;                 // splits > 1: splits x T x m partial sums
    int64_t ldx, ldy, T, n, m;     // n = d_in, m = d_out
    int64_t kper;                  // k per split
    int splits, y_dtype;
    int tiles_t, tiles_m;
};

__device__ __forceinline__ void w8_store(const W8Args& a, int64_t t, int64_t o, float y) {
    const int64_t i = t * a.ldy + o;
    if (a.y_dtype == 0) ((float*)a.Y)[i] = y;
    else ((uint16_t*)a.Y)[i] = a.y_dtype == 1 ? f32_to_f16_bits(y) : f32_to_bf16_bits(y);
}

// One output: the scale of the row first (the sum times it stays inside float32's range), the
// token's last.
__device__ __forceinline__ float w8_value(const W8Args& a, int acc, int64_t t, int64_t o) {
    if (a.zeros) {
        const int z = a.zeros[o];
        acc = (int)((uint32_t)acc + (uint32_t)(128 - (z < 255 ? z : 255)) * (uint32_t)a.sums[t]);
    }
    return ((float)acc * f16_bits_to_f32(a.sw[o])) * a.sx[t];
}

// ------------------------------------------------------------------ any alignment
// 128 x 128 tile, four waves of 64 x 64, 64 k per step, operands through registers into LDS:
// rows may start at any byte and have any length.  A chunk that passes the end of a row is
// assembled from its bytes with 0 past the end (X's zeros make C's bytes there irrelevant).
constexpr int G_TILE = 128, G_BK = 64;

// LDS byte offset of row r's 16-byte chunk c
__device__ __forceinline__ int g_off(int r, int c) { return r * G_BK + 16 * (c ^ ((r >> 1) & 3)); }

__device__ __forceinline__ uint4 g_load(const uint8_t* row, int64_t k, int64_t kend) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (k + 16 <= kend) {
        __builtin_memcpy(&v, row + k, 16);
    } else {
        uint8_t b[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) b[e] = k + e < kend ? row[k + e] : (uint8_t)0;
        __builtin_memcpy(&v, b, 16);
    }
    return v;
}

template <bool ZP>
__global__ __launch_bounds__(256) void w8_any_kernel(W8Args a) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][2 * G_TILE * G_BK];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave & 1, wn = wave >> 1;
    const int64_t t0 = (int64_t)(blockIdx.x % a.tiles_t) * G_TILE;
    const int64_t o0 = (int64_t)(blockIdx.x / a.tiles_t) * G_TILE;
    const int64_t kbeg = (int64_t)blockIdx.y * a.kper;
    const int64_t kend = kbeg + a.kper < a.n ? kbeg + a.kper : a.n;

    // thread t copies the chunk t % 4 of rows t / 4 and 64 + t / 4 of both tiles; rows past the
    // matrices repeat the last one (their outputs are not stored)
    const uint8_t* xr[2];
    const uint8_t* cr[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t r = 64 * q + (tid >> 2);
        xr[q] = (const uint8_t*)a.X + (t0 + r < a.T ? t0 + r : a.T - 1) * a.ldx;
        cr[q] = a.C + (o0 + r < a.m ? o0 + r : a.m - 1) * a.n;
    }
    uint4 xv[2], cv[2];
    auto fetch = [&](int64_t k0) {
        const int64_t k = k0 + 16 * (tid & 3);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            xv[q] = g_load(xr[q], k, kend);
            cv[q] = g_load(cr[q], k, kend);
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int o = g_off(64 * q + (tid >> 2), tid & 3);
            *(uint4*)(lds[buf] + o) = xv[q];
            uint4 c = cv[q];
            if (ZP) { c.x ^= 0x80808080u; c.y ^= 0x80808080u; c.z ^= 0x80808080u; c.w ^= 0x80808080u; }
            *(uint4*)(lds[buf] + G_TILE * G_BK + o) = c;
        }
    };
    i32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
    fetch(kbeg);
    int buf = 0;
    for (int64_t k0 = kbeg; k0 < kend; k0 += G_BK, buf ^= 1) {
        // the other buffer's readers passed the barrier of the step before
        put(buf);
        __syncthreads();
        if (k0 + G_BK < kend) fetch(k0 + G_BK);
        const uint8_t* A = lds[buf];
        const uint8_t* B = A + G_TILE * G_BK;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            i32x4 fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = *(const i32x4*)(A + g_off(wm * 64 + 32 * i + (lane & 31), 2 * ks + (lane >> 5)));
                fb[i] = *(const i32x4*)(B + g_off(wn * 64 + 32 * i + (lane & 31), 2 * ks + (lane >> 5)));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t o = o0 + wn * 64 + 32 * j + (lane & 31);
            if (o >= a.m) continue;
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int64_t t = t0 + wm * 64 + 32 * i + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
                if (t >= a.T) continue;
                if (a.splits > 1) a.part[((int64_t)blockIdx.y * a.T + t) * a.m + o] = acc[i][j][v];
                else w8_store(a, t, o, w8_value(a, acc[i][j][v], t, o));
            }
        }
}

// the splits' sums of each output, scaled
__global__ __launch_bounds__(256) void w8_join_kernel(W8Args a) {
    const int64_t size = a.T * a.m;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < size; i += (int64_t)gridDim.x * 256) {
        uint32_t s = 0;
        for (int k = 0; k < a.splits; ++k) s += (uint32_t)a.part[k * size + i];
        const int64_t t = i / a.m, o = i - t * a.m;
        w8_store(a, t, o, w8_value(a, (int)s, t, o));
    }
}

struct W8Plan {
    int splits;
    int64_t kper;
};

// Splits of k until about two workgroups per compute unit run, each with at least W8_SPLIT_MIN_K
W8Plan w8_plan(int64_t T, int64_t n, int64_t m) {
    const int64_t tiles = cdiv(T, G_TILE) * cdiv(m, G_TILE);
    int64_t s = cdiv(512, tiles);
    if (s > n / W8_SPLIT_MIN_K) s = n / W8_SPLIT_MIN_K;
    if (s < 1) s = 1;
    const int64_t kper = cdiv(cdiv(n, s), G_BK) * G_BK;
    return W8Plan{(int)cdiv(n, kper), kper};
}

}  // namespace

bool w8_size_ok(int64_t T, int64_t n, int64_t m) {
    // work-items of a launch are counted in 32 bits
    return cdiv(T, G_TILE) * cdiv(m, G_TILE) < ((int64_t)1 << 24);
}

size_t w8_ws_bytes(int64_t T, int64_t n, int64_t m) {
    const W8Plan p = w8_plan(T, n, m);
    return p.splits > 1 ? (size_t)p.splits * (size_t)T * (size_t)m * sizeof(int32_t) : 0;
}

hipError_t w8_launch(const int8_t* X, int64_t T, int64_t n, int64_t ldx, const float* sx, const int32_t* sums,
                     const uint8_t* C, const uint16_t* sw, const uint16_t* zeros, int64_t m, void* Y, int y_dtype,
                     int64_t ldy, void* ws, hipStream_t s) {
    const W8Plan p = w8_plan(T, n, m);
    W8Args a{};
    a.X = X; a.sx = sx; a.sums = sums; a.C = C; a.sw = sw; a.zeros = zeros; a.Y = Y; a.part = (int32_t*)ws;
    a.ldx = ldx; a.ldy = ldy; a.T = T; a.n = n; a.m = m; a.kper = p.kper; a.splits = p.splits; a.y_dtype = y_dtype;
    a.tiles_t = (int)cdiv(T, G_TILE); a.tiles_m = (int)cdiv(m, G_TILE);
    const dim3 grid((unsigned)(a.tiles_t * (int64_t)a.tiles_m), (unsigned)p.splits);
    if (zeros) hipLaunchKernelGGL(w8_any_kernel<true>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(w8_any_kernel<false>, grid, dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t blocks = cdiv(T * m, 256);
    hipLaunchKernelGGL(w8_join_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace pwq
