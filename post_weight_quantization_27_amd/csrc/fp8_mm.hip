// Product of e4m3 codes with e4m3 codes, a scale for each block of 128:
//
//   Y[t, o] = sum over blocks b of sx[b, t] sw[o / 128, b] sum over k in b of X[t, k] C[o, k]
//
// and the same grouped by expert: row t belongs to the expert e with offsets[e] <= t < offsets[e + 1],
// multiplies C_e and sw_e, and reads row rows[t] of X (row t without rows).
//
// The matrix instruction on e4m3 operands (K = 128, a block at a time) does not hold its sum in 32
// bits: of each eight consecutive products it keeps what is at least 2^-13 of the largest one's power
// of two (measured: 2^16 + 2^2 gives 2^16).  Codes convert exactly to float16, whose products and sums
// the float16 instruction holds in float32, at half the rate.  So
//   EXACT   float32 outputs, and wherever the weights' traffic is the bound: float16 instructions
//           (error against 64 bits 1.0e-7 of normal data's norm at 8192 inputs);
//   !EXACT  16-bit outputs of tiles, whose own rounding (1.7e-3 of the norm in bfloat16, 2.1e-4 in
//           float16) hides the e4m3 instruction's 1.5e-5 to 5e-5.
// A block's sum is multiplied by its two scales and added to the output's float32 sum.
#include "../../include/pwq.h"
#include "fp8.h"

namespace pwq {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct F8Args {
    const uint8_t* X;
    const void* sx;                // groups x X's rows, pitch ldsx: float32 or e8m0
    const uint8_t* C;              // [experts] d_out x d_in, dense
    const void* sw;                // [experts] d_out / 128 x groups
    const int32_t* offsets;        // experts + 1, or NULL: one matrix for all rows
    const int32_t* rows;           // X's row of each output row, or NULL
    void* Y;
    float* part;                   // splits > 1: splits x T x m partial sums
    int64_t ldx, ldsx, ldy;
    int64_t T, n, m;               // output rows, d_in, d_out
    int64_t xrows, kper;           // X's rows; k per split
    int experts, groups, splits, y_dtype;
    int tiles_t, tiles_m;
};

// ------------------------------------------------------------------ which rows
struct F8Rows {
    int64_t t0, end;               // rows t0 .. end - 1 at most of one expert; none where t0 >= end
    int expert;
};

// Tile tt of BT rows: the experts' rows are cut into tiles one expert after the other.  Every wave
// counts through the offsets, 64 experts at a time.  Offsets are taken into 0 .. T, so whatever they
// hold no row outside Y is touched.
template <int BT>
__device__ __forceinline__ F8Rows f8_rows(const F8Args& a, int tt) {
    if (!a.offsets) return F8Rows{(int64_t)tt * BT, a.T, 0};
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
        int64_t lo = 0, hi = 0;
        if (e0 + lane < a.experts) {
            lo = a.offsets[e0 + lane];
            hi = a.offsets[e0 + lane + 1];
            lo = lo < 0 ? 0 : lo;
            hi = hi > a.T ? a.T : hi;
        }
        const int own = hi > lo ? (int)((hi - lo + BT - 1) / BT) : 0;
        int sum = own;                                    // tiles of the experts up to this one
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(sum, o, 64);
            if (lane >= o) sum += v;
        }
        const uint64_t past = __ballot(before + sum > tt);
        if (past) {
            const int src = __builtin_ctzll(past);
            const int64_t t0 = lo + (int64_t)(tt - before - (sum - own)) * BT;
            F8Rows r;
            r.t0 = ((int64_t)__builtin_amdgcn_readlane((int)(t0 >> 32), src) << 32) |
                   (uint32_t)__builtin_amdgcn_readlane((int)t0, src);
            r.end = ((int64_t)__builtin_amdgcn_readlane((int)(hi >> 32), src) << 32) |
                    (uint32_t)__builtin_amdgcn_readlane((int)hi, src);
            r.expert = e0 + src;
            return r;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return F8Rows{0, 0, 0};
}

// X's row for output row t; bad indexes read row 0 and give NaN (f8_bad)
__device__ __forceinline__ int64_t f8_xrow(const F8Args& a, int64_t t) {
    if (!a.rows) return t;
    const int64_t r = a.rows[t];
    return r >= 0 && r < a.xrows ? r : 0;
}
__device__ __forceinline__ bool f8_bad(const F8Args& a, int64_t t) {
    return a.rows && (uint32_t)a.rows[t] >= (uint64_t)a.xrows;
}

// bid -> tile: consecutive workgroups go to different XCDs, so each XCD takes a contiguous share
// of the tiles, in groups of up to 8 output tiles by all token tiles
__device__ __forceinline__ void f8_map(const F8Args& a, int64_t bid, int& to, int& tt) {
    const int64_t nt = (int64_t)a.tiles_t * a.tiles_m;
    const int64_t x = bid & 7, per = nt >> 3, rem = nt & 7;
    const int64_t id = x * per + (x < rem ? x : rem) + (bid >> 3);
    const int64_t band = 8 * (int64_t)a.tiles_t, g = id / band;
    const int rows = a.tiles_m - 8 * g < 8 ? (int)(a.tiles_m - 8 * g) : 8;
    const int in = (int)(id - g * band);
    tt = in / rows;
    to = (int)(8 * g) + in - tt * rows;
}

// ------------------------------------------------------------------ scales
template <bool E8>
__device__ __forceinline__ float f8_get(const void* s, int64_t i) {
    if constexpr (E8) {
        const uint32_t b = ((const uint8_t*)s)[i];       // 2^(b - 127); 0 is below the normal floats, 255 NaN
        return __builtin_bit_cast(float, b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
    } else {
        return ((const float*)s)[i];
    }
}
// index of the scale of outputs o (within one block) and block b
__device__ __forceinline__ int64_t f8_sw_at(const F8Args& a, int expert, int64_t o, int64_t b) {
    return ((int64_t)expert * ((a.m + F8_B - 1) / F8_B) + (o < a.m ? o : a.m - 1) / F8_B) * a.groups + b;
}

// ------------------------------------------------------------------ codes
// eight codes as float16, exactly
__device__ __forceinline__ f16x8 f8_half(int lo, int hi) {
    f16x8 v;
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
    v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
    v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
    return v;
}

// ------------------------------------------------------------------ outputs
__device__ __forceinline__ uint16_t f8_16(const F8Args& a, float y) {
    return a.y_dtype == 1 ? f32_to_f16_bits(y) : f32_to_bf16_bits(y);
}
// outputs o .. o + 3 of row t, as far as they are there, in one piece at any address
__device__ __forceinline__ void f8_put4(const F8Args& a, f32x4 y, int64_t t, int64_t o) {
    const int64_t i = t * a.ldy + o;
    if (a.y_dtype == 0) {
        float* p = (float*)a.Y + i;
        if (o + 4 <= a.m) {
            __builtin_memcpy(p, &y, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (o + e < a.m) p[e] = y[e];
        }
    } else {
        uint16_t* p = (uint16_t*)a.Y + i;
        uint16_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = f8_16(a, y[e]);
        if (o + 4 <= a.m) {
            __builtin_memcpy(p, v, 8);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (o + e < a.m) p[e] = v[e];
        }
    }
}
// the same, or the sums over this split of k
__device__ __forceinline__ void f8_out4(const F8Args& a, f32x4 y, int64_t t, int64_t end, int64_t o, bool bad) {
    if (o >= a.m || t >= end) return;
    if (bad) y = (f32x4){__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
    if (a.splits > 1) {
        float* p = a.part + ((int64_t)blockIdx.y * a.T + t) * a.m + o;
        if (o + 4 <= a.m) {
            __builtin_memcpy(p, &y, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (o + e < a.m) p[e] = y[e];
        }
        return;
    }
    f8_put4(a, y, t, o);
}

// ------------------------------------------------------------------ waits
// all LDS reads and writes of this wave are done
__device__ __forceinline__ void f8_wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }
// workgroup barrier without a fence: loads stay in flight across it
__device__ __forceinline__ void f8_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
// position of 16-byte chunk c in row r of a stage of 128-byte rows: the 16 lanes that a 16-byte LDS
// read serves at a time hit 16 different bank groups
__device__ __forceinline__ int f8_pos(int r, int c) { return c ^ ((r >> 1) & 7); }

// ------------------------------------------------------------------ any alignment
// BO x BT tile (outputs x tokens), four waves as 2 x 2, a block of 128 k per step: rows may start at
// any byte and have any length.  Operands travel through registers into LDS, two steps ahead; LDS
// has two buffers and a step one barrier.  The last step may be partial: each 16 bytes past the end
// is the row's last 16 instead, moved down in registers, with 0 behind in both operands (a byte
// from elsewhere may be NaN).

// The 16 bytes from byte `by` (0 .. 16) on, with 0 behind them
__device__ __forceinline__ uint4 f8_drop(uint4 v, int by) {
    if (by & 16) v = make_uint4(0u, 0u, 0u, 0u);
    if (by & 8) v = make_uint4(v.z, v.w, 0u, 0u);
    if (by & 4) v = make_uint4(v.y, v.z, v.w, 0u);
    const uint32_t b = (uint32_t)by & 3u;
    return make_uint4(__builtin_amdgcn_alignbyte(v.y, v.x, b), __builtin_amdgcn_alignbyte(v.z, v.y, b),
                      __builtin_amdgcn_alignbyte(v.w, v.z, b), __builtin_amdgcn_alignbyte(0u, v.w, b));
}

// 16 bytes of a row shorter than 16, from its byte k on, with 0 past its n
__device__ __forceinline__ uint4 f8_short(const uint8_t* row, int64_t k, int64_t n) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int e = 0; e < 16 && k + e < n; ++e) {
        const uint32_t byte = (uint32_t)row[k + e] << (8 * (e & 3));
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] |= c == e / 4 ? byte : 0u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int BO, int BT, int P, bool E8>
__global__ __launch_bounds__(256) void f8_any_kernel(F8Args a) {
    constexpr int BK = F8_B, FO = BO / 32, FT = BT / 32;      // fragments of a wave
    constexpr int NC = (BO + BT) / 32;                        // chunks per thread
    constexpr int ST = (BO + BT) * BK;
    static_assert(BO <= 256, "a wave's outputs share a block");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * ST];
    int to, tt;
    f8_map(a, blockIdx.x, to, tt);
    const F8Rows at_rows = f8_rows<BT>(a, tt);
    if (at_rows.t0 >= at_rows.end) return;
    const int64_t o0 = (int64_t)to * BO, t0 = at_rows.t0, tend = at_rows.end;
    const int64_t kbeg = (int64_t)blockIdx.y * a.kper;
    const int64_t kend = kbeg + a.kper < a.n ? kbeg + a.kper : a.n;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wo = wave & 1, wt = wave >> 1;

    // chunk j of this thread: chunk tid % 8 of row j 32 + tid / 8 of the codes' BO rows followed by
    // the activations' BT; rows past the matrices repeat the last one (not stored)
    const uint8_t* src[NC];
    int dst[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int r = j * 32 + (tid >> 3);
        if (r < BO) src[j] = a.C + ((int64_t)at_rows.expert * a.m + (o0 + r < a.m ? o0 + r : a.m - 1)) * a.n;
        else src[j] = a.X + f8_xrow(a, t0 + r - BO < tend ? t0 + r - BO : tend - 1) * a.ldx;
        dst[j] = r * BK + 16 * f8_pos(r & 15, tid & 7);
    }
    const int r = lane & 15, c = lane >> 4;
    const int64_t ob = o0 + wo * (BO / 2), tb = t0 + wt * (BT / 2) + r;
    int64_t xs[FT];                                           // X's rows of this lane's tokens
#pragma unroll
    for (int j = 0; j < FT; ++j) xs[j] = f8_xrow(a, tb + 16 * j < tend ? tb + 16 * j : tend - 1);
    const int64_t wat = f8_sw_at(a, at_rows.expert, ob, 0);
    const int nsteps = (int)cdiv(kend - kbeg, BK), nfull = (int)((kend - kbeg) / BK);
    auto at = [&](int it) {                                   // the step's k here, no later than the last 16 bytes
        const int64_t k = kbeg + (int64_t)(it < nsteps ? it : nsteps - 1) * BK + 16 * (tid & 7);
        return k < kend - 16 ? k : kend - 16;
    };
    struct Step {
        uint4 v[NC];
        float sx[FT], sw;
    };
    auto scales = [&](Step& s, int it) {
        const int64_t b = kbeg / BK + (it < nsteps ? it : nsteps - 1);
#pragma unroll
        for (int j = 0; j < FT; ++j) s.sx[j] = f8_get<E8>(a.sx, b * a.ldsx + xs[j]);
        s.sw = f8_get<E8>(a.sw, wat + b);
    };
    auto fetch = [&](Step& s, int it) {
        const int64_t k = at(it);
#pragma unroll
        for (int j = 0; j < NC; ++j) __builtin_memcpy(&s.v[j], src[j] + k, 16);
        scales(s, it);
    };
    f32x4 acc[FO][FT];
#pragma unroll
    for (int i = 0; i < FO; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const uint8_t* S, const float (&sx)[FT], float sw) {
        f8_wait_lds();
        f8_barrier();
        f32x4 p[FO][FT];
#pragma unroll
        for (int i = 0; i < FO; ++i)
#pragma unroll
            for (int j = 0; j < FT; ++j) p[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < BK / 64; ++ks) {
            const int o = r * BK + 16 * f8_pos(r, 4 * ks + c);
            i32x4 fo[FO], ft[FT];
#pragma unroll
            for (int i = 0; i < FO; ++i) fo[i] = *(const i32x4*)(S + (wo * (BO / 2) + 16 * i) * BK + o);
#pragma unroll
            for (int j = 0; j < FT; ++j) ft[j] = *(const i32x4*)(S + (BO + wt * (BT / 2) + 16 * j) * BK + o);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f16x8 ho[FO], ht[FT];
#pragma unroll
                for (int i = 0; i < FO; ++i) ho[i] = f8_half(fo[i][2 * h], fo[i][2 * h + 1]);
#pragma unroll
                for (int j = 0; j < FT; ++j) ht[j] = f8_half(ft[j][2 * h], ft[j][2 * h + 1]);
#pragma unroll
                for (int i = 0; i < FO; ++i)
#pragma unroll
                    for (int j = 0; j < FT; ++j) p[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ho[i], ht[j], p[i][j], 0, 0, 0);
            }
        }
#pragma unroll
        for (int j = 0; j < FT; ++j) {
            const float s = sx[j] * sw;
#pragma unroll
            for (int i = 0; i < FO; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[i][j][e], s, acc[i][j][e]);
        }
    };
    // step `it` (a whole one: 128 k), whose chunks are in s; s is refilled for a later one under its
    // products
    auto step = [&](Step& s, int it, int next) {
        uint8_t* S = lds + (it & 1) * ST;
        float sx[FT];
        const float sw = s.sw;
#pragma unroll
        for (int j = 0; j < FT; ++j) sx[j] = s.sx[j];
#pragma unroll
        for (int j = 0; j < NC; ++j) *(uint4*)(S + dst[j]) = s.v[j];
        fetch(s, next);
        multiply(S, sx, sw);
    };
    auto last = [&](Step& s, int it) {                        // one of the last, nothing to fetch
        uint8_t* S = lds + (it & 1) * ST;
        const int64_t drop = kbeg + (int64_t)it * BK + 16 * (tid & 7) - at(it);
#pragma unroll
        for (int j = 0; j < NC; ++j) *(uint4*)(S + dst[j]) = it < nfull ? s.v[j] : f8_drop(s.v[j], (int)(drop < 16 ? drop : 16));
        multiply(S, s.sx, s.sw);
    };
    if (a.n >= 16) {
        Step s[P];
#pragma unroll
        for (int u = 0; u < P; ++u) fetch(s[u], u);
        int it = 0;
        for (; it + P <= nfull; it += P) {
#pragma unroll
            for (int u = 0; u < P; ++u) step(s[u], it + u, it + u + P);
        }
#pragma unroll
        for (int u = 0; u < P; ++u)
            if (it + u < nsteps) last(s[u], it + u);
    } else {                                                  // one step
        Step s;
        scales(s, 0);
#pragma unroll
        for (int j = 0; j < NC; ++j) *(uint4*)(lds + dst[j]) = f8_short(src[j], 16 * (tid & 7), a.n);
        multiply(lds, s.sx, s.sw);
    }
#pragma unroll
    for (int j = 0; j < FT; ++j) {
        const int64_t t = tb + 16 * j;
        const bool bad = t < tend && f8_bad(a, t);
#pragma unroll
        for (int i = 0; i < FO; ++i) f8_out4(a, acc[i][j], t, tend, ob + 16 * i + 4 * c, bad);
    }
}

// ------------------------------------------------------------------ launches
template <int BO, int BT, int P>
hipError_t f8_any_go(F8Args a, bool e8, hipStream_t s) {
    a.tiles_m = (int)cdiv(a.m, BO);
    // an expert's last tile may be partial: one more tile for each that has rows, at most
    a.tiles_t = (int)(a.offsets ? a.T / BT + (a.T < a.experts ? a.T : a.experts) : cdiv(a.T, BT));
    const dim3 grid((unsigned)(a.tiles_m * (int64_t)a.tiles_t), (unsigned)a.splits);
    if (e8) hipLaunchKernelGGL((f8_any_kernel<BO, BT, P, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((f8_any_kernel<BO, BT, P, false>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

bool f8_size_ok(int64_t T, int64_t m, int64_t experts) {
    // work-items of a launch are counted in 32 bits: 512 for each tile of 64 x 16 at least
    return (cdiv(T, 64) + (T < experts ? T : experts)) * cdiv(m, 64) < ((int64_t)1 << 23);
}
size_t f8_ws_bytes(int64_t T, int64_t n, int64_t m, int64_t experts) {
    (void)T; (void)n; (void)m; (void)experts;
    return 0;
}

hipError_t f8_launch(const F8Call& c, hipStream_t s) {
    F8Args a{};
    a.X = c.X; a.sx = c.sx; a.C = c.C; a.sw = c.sw; a.offsets = c.offsets; a.rows = c.rows; a.Y = c.Y;
    a.part = (float*)c.ws; a.ldx = c.ldx; a.ldsx = c.ldsx; a.ldy = c.ldy; a.T = c.T; a.n = c.n; a.m = c.m;
    a.xrows = c.xrows; a.experts = (int)c.experts; a.groups = (int)cdiv(c.n, F8_B); a.y_dtype = c.y_dtype;
    a.splits = 1;
    a.kper = c.n;
    return f8_any_go<64, 64, 2>(a, c.e8, s);
}

}  // namespace pwq
