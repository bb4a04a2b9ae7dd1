// Product of e4m3 codes with e4m3 codes, a scale for each block of 128:
//
//   Y[t, o] = sum over blocks b of sx[b, t] sw[o / 128, b] sum over k in b of X[t, k] C[o, k]
//
// and the same grouped by expert: row t belongs to the expert e with offsets[e] <= t < offsets[e + 1],
// multiplies C_e and sw_e, and reads row rows[t] of X (row t without rows).
//
// The matrix instruction on e4m3 operands (K = 128, a block at a time) does not hold its sum in 32
// bits: of each eight consecutive products it keeps what is at least 2^-13 of the largest one's power
// of two (measured: 2^16 + 2^2 gives 2^16), so large products that cancel can take a result with them.
// Codes convert exactly to float16, whose products and sums the float16 instruction holds in float32, at
// half the rate.  So
//   EXACT   whatever the output's type: float16 instructions (error against 64 bits 1.0e-7 of normal
//           data's norm at 8192 inputs).  The row kernel and the joins of splits have no other form;
//   !EXACT  tiles whose 16-bit outputs the caller asks for with PWQ_E4M3_SUMS: the e4m3 instruction, off
//           by 1.5e-5 to 5e-5 of normal data's norm, beside the output's own rounding (1.7e-3 in bfloat16,
//           2.1e-4 in float16).
// A block's sum is multiplied by its two scales and added to the output's float32 sum; powers of two with
// !EXACT go into the instruction, which adds the block to the sum itself.
#include "../../include/pwq.h"
#include "fp8.h"
#include "fp8_plan.h"

#include <type_traits>

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
    int tiles_t, tiles_m;          // launched
    bool laid;                     // X is a copy, a row for each output row
};

// ------------------------------------------------------------------ which rows
struct F8Rows {
    int64_t t0, end;               // rows t0 .. end - 1 at most of one expert; none where t0 >= end
    int expert;
};

// The experts' rows are cut into tiles of BT, one expert after the other.  Every wave counts them through
// the offsets, 64 experts at a time.  Offsets are taken into 0 .. T, and a tile has to start inside its
// expert's rows, and no more tiles count than were launched, so whatever the offsets hold no row outside Y is
// touched and no output outside 0 .. d_out - 1.
template <int BT>
struct F8Count {
    int64_t lo, hi;                // of this lane's expert
    int own, upto;                 // its tiles, and those of the experts up to it (of the same 64)
    __device__ __forceinline__ int of(const F8Args& a, int e0) {      // tiles of the 64 experts from e0 on
        const int lane = threadIdx.x & 63;
        lo = hi = 0;
        if (e0 + lane < a.experts) {
            lo = f8_low(a.offsets[e0 + lane]);
            hi = f8_high(a.offsets[e0 + lane + 1], a.T);
        }
        own = f8_own(lo, hi, BT, a.tiles_t);
        upto = own;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o, 64);
            if (lane >= o) upto += v;
        }
        return __builtin_amdgcn_readlane(upto, 63);
    }
    // the rows of tile tt of these 64 experts, if it is one of theirs
    __device__ __forceinline__ bool find(int e0, int tt, F8Rows& r) const {
        const uint64_t past = __ballot(upto > tt);
        if (!past) return false;
        const int src = __builtin_ctzll(past);
        const int64_t t = lo + (int64_t)(tt - (upto - own)) * BT, t0 = t >= lo && t < hi ? t : hi;
        r.t0 = ((int64_t)__builtin_amdgcn_readlane((int)(t0 >> 32), src) << 32) | (uint32_t)__builtin_amdgcn_readlane((int)t0, src);
        r.end = ((int64_t)__builtin_amdgcn_readlane((int)(hi >> 32), src) << 32) | (uint32_t)__builtin_amdgcn_readlane((int)hi, src);
        r.expert = e0 + src;
        return true;
    }
};

// Tile tt of BT rows
template <int BT>
__device__ __forceinline__ F8Rows f8_rows(const F8Args& a, int tt) {
    if (!a.offsets) return F8Rows{(int64_t)tt * BT, a.T, 0};
    F8Rows r{0, 0, 0};
    F8Count<BT> c;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
        const int n = c.of(a, e0);
        if (c.find(e0, tt, r)) break;
        tt -= n;
    }
    return r;
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

// bid -> tile of BT rows by outputs (f8_place).  With experts the XCDs' shares are of the tiles that hold
// rows: of those that might, which are launched, the last ones hold none (32768 rows of 64 experts by 4096 x
// 4096, PWQ_E4M3_SUMS: 708 us with shares of all, 609 so).
template <int BT>
__device__ __forceinline__ bool f8_tile(const F8Args& a, uint32_t bid, int& to, F8Rows& r) {
    F8Count<BT> c;
    uint32_t tiles_t = (uint32_t)a.tiles_t;
    if (a.offsets) {
        tiles_t = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 64) tiles_t = f8_upto(tiles_t, c.of(a, e0), a.tiles_t);
    }
    const F8Place p = f8_place(bid, tiles_t, (uint32_t)a.tiles_m);
    if (!p.there) return false;
    to = p.to;
    if (a.offsets && a.experts <= 64) c.find(0, p.tt, r);
    else r = f8_rows<BT>(a, p.tt);
    return r.t0 < r.end;
}

// ------------------------------------------------------------------ scales
// 2^(b - 127); 0 is below the normal floats, 255 NaN
__device__ __forceinline__ float f8_pow2(uint32_t b) {
    return __builtin_bit_cast(float, b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
}
template <bool E8>
__device__ __forceinline__ float f8_get(const void* s, int64_t i) {
    if constexpr (E8) {
        return f8_pow2(((const uint8_t*)s)[i]);
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
// Two fragments' outputs in 16 bits, o0 .. o0 + 31 of the 16 rows that a wave's lanes hold (lane row
// c: outputs 4 c .. 4 c + 3 of each fragment).  Two swaps between lane rows give row c the outputs 8 c
// .. 8 c + 7, so that a store writes 64 bytes of a row in one piece instead of 32.
__device__ __forceinline__ void f8_put_pair16(const F8Args& a, f32x4 y0, f32x4 y1, int64_t t, int64_t end, int64_t o0, int c,
                                              bool bad) {
    uint32_t even[2], odd[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto s = __builtin_amdgcn_permlane32_swap((uint32_t)f8_16(a, y0[2 * h]) | ((uint32_t)f8_16(a, y0[2 * h + 1]) << 16),
                                                        (uint32_t)f8_16(a, y1[2 * h]) | ((uint32_t)f8_16(a, y1[2 * h + 1]) << 16),
                                                        false, false);
        const auto r = __builtin_amdgcn_permlane16_swap(s[0], s[1], false, false);
        even[h] = r[0];
        odd[h] = r[1];
    }
    const uint32_t nan = 0x7fc07fc0u;                     // a NaN in both 16-bit types
    const uint32_t v[4] = {bad ? nan : even[0], bad ? nan : even[1], bad ? nan : odd[0], bad ? nan : odd[1]};
    const int64_t o = o0 + 8 * c;
    if (o >= a.m || t >= end) return;
    uint16_t* p = (uint16_t*)a.Y + t * a.ldy + o;
    if (o + 8 <= a.m) {
        __builtin_memcpy(p, v, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (o + e < a.m) p[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
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
// from elsewhere may be NaN).  Loads at odd addresses and the conversions to float16 bound it: 2000 rows by
// 8191 x d_in, bfloat16, 530 us with d_in 8191, 453 with 8196 and 440 with 8192, and the tiles below 234; with
// PWQ_E4M3_SUMS 360, 281, 244 and 120.

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

template <int BO, int BT, int P, bool E8, bool EXACT>
__global__ __launch_bounds__(256) void f8_any_kernel(F8Args a) {
    constexpr int BK = F8_B, FO = BO / 32, FT = BT / 32;      // fragments of a wave
    constexpr int NC = (BO + BT) / 32;                        // chunks per thread
    constexpr int ST = (BO + BT) * BK;
    static_assert(BO <= 256, "a wave's outputs share a block");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * ST];
    int to;
    F8Rows at_rows{0, 0, 0};
    if (!f8_tile<BT>(a, blockIdx.x, to, at_rows)) return;
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
    auto read = [&](const uint8_t* S, int row) {              // this lane's chunks c and c + 4 of row + r
        const uint8_t* q = S + (row + r) * BK;
        const i32x4 u = *(const i32x4*)(q + 16 * f8_pos(r, c)), v = *(const i32x4*)(q + 16 * f8_pos(r, 4 + c));
        return __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto multiply = [&](const uint8_t* S, const float (&sx)[FT], float sw) {
        f8_wait_lds();
        f8_barrier();
        f32x4 p[FO][FT];
        i32x8 fo[FO], ft[FT];
#pragma unroll
        for (int i = 0; i < FO; ++i) fo[i] = read(S, wo * (BO / 2) + 16 * i);
#pragma unroll
        for (int j = 0; j < FT; ++j) ft[j] = read(S, BO + wt * (BT / 2) + 16 * j);
#pragma unroll
        for (int i = 0; i < FO; ++i)
#pragma unroll
            for (int j = 0; j < FT; ++j) p[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
        if constexpr (EXACT) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
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
        } else {
#pragma unroll
            for (int i = 0; i < FO; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j)
                    p[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fo[i], ft[j], p[i][j], 0, 0, 0, 0, 0, 0);
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

// ------------------------------------------------------------------ rows of 16-byte multiples
// BO x BT tile (outputs x tokens), eight waves, a block of 128 k per stage; the codes are the row
// operand, so that a lane ends with four consecutive outputs of one token.
//
// Operand rows go straight from memory into LDS (global_load_lds, 16 bytes a lane), and so do the
// block's scales, four bytes a lane: the tokens' and behind them the outputs'.  A row's 16-byte chunk
// c lies at f8_pos, which keeps the reads free of bank conflicts.  A lane's operand of the e4m3
// instruction is its row's chunks c and c + 4: any order of k will do that both operands share.
//
// The waves work in two groups of four, one half step apart: while one group reads its fragments of
// a stage, the other runs its matrix instructions and adds the block's sums to its outputs', with a
// barrier between the half steps.  Each SIMD holds one wave of each group.
//   KG = 1: both groups take every stage, each its half of the tile (WO x 8 / WO waves).
//   KG = 2: each group takes every other stage for the whole tile (WO x 4 / WO waves), with stages of
//           its own that its own waves copy; the two sums meet in LDS at the end.
// NST stages: a stage's copies fly while the NST - 1 before it are used.  With two (256 x 256, whose
// stages are 64 KB) the step is cut in two, each with its half of the wave's rows, so that half a step's
// fragments are held at a time, and each part of a stage is copied over as soon as it has been read (see the
// loop).
//
// Measured (kernel trace, operands cold, bfloat16 outputs): 8192^3 871-892 us (1.23-1.26 PFLOP/s on the
// float16 instructions, whose library product reaches 1.48), 8192 rows by 28672 x 8192 3000-3160, in tiles of
// 256 x 128: twice as many converted rows do not fit the registers.  With PWQ_E4M3_SUMS, in tiles of 256 x
// 256, 8192^3 419-422 us and 8192 rows by 28672 x 8192 1455-1500 with float32 scales (2.6 PFLOP/s), 373-387
// and 1325-1370 with powers of two (2.8-2.9), where the library's product with one scale per tensor takes
// 1200-1330 on the same boards.  The clock falls to 1.6-2.0 GHz; a step of 256 x 256 takes 2340 cycles with
// powers of two and about 3000 with float32 scales, of 2048 that its instructions need.  Of a tile's time 1.7
// us go before its first copy, 1.4 to 2 until that has landed and 3 to 4 into the outputs (32 steps of 4096
// inputs: 45).
//
// The kernels of 256 x 256 take all 256 registers and spill 11 to 39 more, in the set-up and the loops of the
// last stages: 8192 rows by 28672 x 8192 write 595 MB with powers of two and 510 with float32 scales, for 470
// of outputs.  Workgroups that go through several tiles, whose next addresses take registers too, lose (8192^3
// 5 %, with more spilled; 128 x 128, 300 rows by 50304 x 768 45 us in place of 40), as does leaving out the
// instructions of waves without tokens (1460 -> 1560).
typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ const uint4 f8_zeros = {0u, 0u, 0u, 0u};

// s_waitcnt with only the vector-memory count constrained: vmcnt <= N
template <int N>
__device__ __forceinline__ void f8_wait_vm() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// A buffer from `base` on, for loads at 32-bit offsets: a lane's own and one for all.  The kernels keep
// inside the operands; the size says only that any offset will do.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t f8_buffer(const uint8_t* base) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, -1, 0x00027000);
}

template <int BO, int BT, int NST, int KG>
constexpr int f8_smem = KG * NST * ((BO + BT) * F8_B + 8 / KG * 256);

template <int BO, int BT, int NST, int WO, int KG, bool E8, bool EXACT>
__device__ __forceinline__ void f8_tile_body(const F8Args& a, uint8_t* smem, int to, const F8Rows& at) {
    constexpr int BK = F8_B, NW = 8 / KG, WT = NW / WO;   // waves that share a stage
    constexpr int FO = BO / WO / 16, FT = BT / WT / 16;
    constexpr int FP = NST == 2 ? FO / 2 : FO;            // rows of fragments in registers at a time
    constexpr int Q = FP * FT;                            // tiles of 16 x 16 of a part
    constexpr int L = (BO + BT) / 8 / NW;                 // copies of 8 rows per wave and stage, and one of scales
    constexpr bool TWO = NST == 2;
    constexpr int SLOT = (BO + BT) * BK, ST = SLOT + NW * 256;
    constexpr int NB = BO > F8_B ? BO / F8_B : 1;         // blocks of outputs
    static_assert(L * NW * 8 == BO + BT && BO % (NW * 8) == 0 && (L + 1) * (NST - 1) < 64 && KG * NST * ST <= 163840, "tile");
    static_assert(BO / WO <= F8_B && BT % 64 == 0 && BT / 64 < NW, "scales");
    static_assert(KG == 1 || (NST > 2 && FO % 2 == 0 && 8 * FO / 2 * FT * 1024 <= 2 * NST * ST), "the groups' sums fit the stages");
    static_assert(KG * NST * ST == f8_smem<BO, BT, NST, KG>, "stages");
    const int lane = threadIdx.x & 63, wave8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = KG == 2 ? wave8 & 3 : wave8, grp = wave8 >> 2;
    const int wo = wave / WT, wt = wave % WT;
    uint8_t* const lds = smem + (KG == 2 ? grp * (NST * ST) : 0);
    // this wave's k: from kbeg in steps of KG BK; nk of its stages, the first nfull of which end
    // inside the rows; nmax steps for everybody
    const int64_t kend = (blockIdx.y + 1) * a.kper < a.n ? (blockIdx.y + 1) * a.kper : a.n;
    const int64_t kbeg = (int64_t)blockIdx.y * a.kper + (KG == 2 ? grp * BK : 0);
    const int64_t klen = kend - kbeg;
    const int nk = klen > 0 ? (int)((klen + KG * BK - 1) / (KG * BK)) : 0;
    const int nfull = klen >= BK ? (int)((klen - BK) / (KG * BK)) + 1 : 0;
    const int nmax = KG == 2 ? (int)((kend - (int64_t)blockIdx.y * a.kper + KG * BK - 1) / (KG * BK)) : nk;

    // copy j of this wave: 8 rows from row0(j) on, of the codes' BO rows followed by the activations' BT;
    // a lane brings the chunk that its position holds, from an offset (32 bits) past the operand's base.
    // Rows past the matrices repeat the last one (their outputs are not stored).  One more copy brings
    // 64 scales: the tokens' (slots 0 ..) or the outputs'.
    auto row0 = [&](int j) {
        if constexpr (TWO) {
            // the first group brings codes, rows 0 .. 63 of both halves and then the others; the second X
            if (wave < 4) return (wave >> 1) * 128 + (j >= 4 ? 64 : 0) + (wave & 1) * 32 + (j & 3) * 8;
            return BO + (j >= 4 ? 128 : 0) + (wave - 4) * 32 + (j & 3) * 8;
        }
        return (j * NW + wave) * 8;
    };
    auto of_x = [&](int j) { return TWO ? grp == 1 : j * NW * 8 >= BO; };
    const int slot = TWO ? (wave + 4) & 7 : wave;
    const uint8_t* xbase;
    const uint8_t* cbase;
    __amdgpu_buffer_rsrc_t xbuf, cbuf;
    const uint8_t* sbase;
    int64_t sstep;
    uint32_t off[L];
    const int64_t o0 = (int64_t)to * BO;
    // The order of k is free, so tiles that live on the codes' traffic start at different k: where d_in
    // is a multiple of 4096, rows that are read at the same k in step all come from the same few
    // memory channels.  Large token tiles share X by k instead and start together.
    constexpr int ROT = BT <= 128 ? 3 : 0;
    const int rot = ROT && nfull > 0 ? (int)((uint32_t)(to * ROT) % (uint32_t)nfull) : 0;
    cbase = a.C + ((int64_t)at.expert * a.m + o0) * a.n + kbeg;
    xbase = a.X + (a.rows && !a.laid ? 0 : at.t0 * a.ldx) + kbeg;
    cbuf = f8_buffer(TWO && grp == 1 ? xbase : cbase);
    xbuf = f8_buffer(xbase);                          // two stages: a wave copies rows of one operand alone, cbuf's
#pragma unroll
    for (int j = 0; j < L; ++j) {
        const int r = row0(j) + (lane >> 3);
        const int ch = f8_pos(r & 15, lane & 7);      // the xor undoes itself
        if (of_x(j)) {
            const int64_t t = at.t0 + r - BO < at.end ? at.t0 + r - BO : at.end - 1;
            off[j] = (uint32_t)((a.rows && !a.laid ? f8_xrow(a, t) : t - at.t0) * a.ldx + 16 * ch);
        } else {
            off[j] = (uint32_t)((o0 + r < a.m ? r : a.m - 1 - o0) * a.n + 16 * ch);
        }
    }
    constexpr int SB = E8 ? 1 : 4;
    const int64_t b = kbeg / BK;
    if (slot < BT / 64) {
        const int64_t t = at.t0 + 64 * slot + lane < at.end ? at.t0 + 64 * slot + lane : at.end - 1;
        sbase = (const uint8_t*)a.sx + (b * a.ldsx + f8_xrow(a, t)) * SB;
        sstep = a.ldsx * SB;
    } else {
        sbase = (const uint8_t*)a.sw + f8_sw_at(a, at.expert, o0 + F8_B * (lane % NB), b) * SB;
        sstep = SB;
    }
    // copy j of stage `it` (j = L: the scales).  END: the last stage where it ends past the rows: zeros
    // there in both operands (a byte from elsewhere may be NaN)
    auto copy = [&](auto end, int it, int j) {
        constexpr bool END = decltype(end)::value;
        uint8_t* S = lds + (it % NST) * ST;
        const int pos = !END && ROT ? (it + rot >= nfull ? it + rot - nfull : it + rot) : it;
        if (TWO) j = j < 4 ? j : j == 4 ? L : j - 1;          // the scales with the first four
        if (j == L) {
            const uint8_t* p = sbase + (int64_t)pos * KG * sstep;
            if constexpr (E8) __builtin_amdgcn_global_load_lds((const void*)p, (lds_ptr_t)(S + SLOT + slot * 256), 1, 0, 0);
            else __builtin_amdgcn_global_load_lds((const void*)p, (lds_ptr_t)(S + SLOT + slot * 256), 4, 0, 0);
        } else if constexpr (END) {
            const int64_t k = (int64_t)it * (KG * BK);
            const int ch = f8_pos((row0(j) + (lane >> 3)) & 15, lane & 7);
            const uint8_t* base = (of_x(j) ? xbase : cbase) + k;
            const uint8_t* p = kbeg + k + 16 * ch < kend ? base + off[j] : (const uint8_t*)&f8_zeros;
            __builtin_amdgcn_global_load_lds((const void*)p, (lds_ptr_t)(S + row0(j) * BK), 16, 0, 0);
        } else {
            if (!TWO && of_x(j))
                __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (lds_ptr_t)(S + row0(j) * BK), 16, (int)off[j], pos * (KG * BK), 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(cbuf, (lds_ptr_t)(S + row0(j) * BK), 16, (int)off[j], pos * (KG * BK), 0, 0);
        }
    };
    using No = std::false_type;
    using Yes = std::true_type;
    auto copy_some = [&](int it, int from, int to) {      // copies from .. to - 1, of a stage that may not be
        for (int j = from; j < to; ++j) {
            if (it < nfull) copy(No{}, it, j);
            else if (it < nk) copy(Yes{}, it, j);
        }
    };

    f32x4 acc[FO][FT];
    const int r = lane & 15, c = lane >> 4;
    const uint8_t* la[2];
    const uint8_t* lb[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int o = r * BK + 16 * f8_pos(r, 4 * h + c);
        la[h] = lds + wo * (BO / WO) * BK + o;
        lb[h] = lds + (BO + wt * (BT / WT)) * BK + o;
    }
    const uint8_t* const ls = lds + SLOT + 4 * (wt * (BT / WT) + r);
    const uint8_t* const lw = lds + SLOT + 4 * (BT + wo * (BO / WO) / F8_B);
    // A part of the wave's FO rows of fragments against all of its tokens, whose fragments and scales the
    // first part reads.  `read`: what else the half step of the reads does; `during(q)`: what the other
    // does behind matrix instruction q.
    //
    // Scales of powers of two go into the e4m3 instruction, which adds to the outputs' sums itself.
    // Otherwise a tile's block sum is added AHEAD instructions after the one that makes it: a wave's vector
    // instructions run under its own matrix instructions only in part (32 cycles an instruction alone,
    // 40 with its four multiply-adds, 45 where the last results are waited for).  With two stages the last
    // AHEAD of a part are added in the next half step of reads (`rest`), which has time for it.
    constexpr bool INSIDE = E8 && !EXACT;                 // the scales are the instruction's
    constexpr int AHEAD = 2;
    i32x8 ft[FT];
    uint32_t sx[FT], sw;
    float s[FT];
    f32x4 p[AHEAD + 1];
    auto add = [&](int i0, int q, const f32x4& v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i0 + q / FT][q % FT][e] = __builtin_fmaf(v[e], s[q % FT], acc[i0 + q / FT][q % FT][e]);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto rest = [&](int i0) {                             // of the part before the one from row i0 on
        if constexpr (!INSIDE && TWO) {
#pragma unroll
            for (int q = Q - AHEAD; q < Q; ++q) add(i0 ? 0 : FO - FP, q, p[q % (AHEAD + 1)]);
        }
    };
    auto step = [&](auto part, int it, auto read, auto during) {
        constexpr int I0 = decltype(part)::value * FP;
        const int st = (it % NST) * ST;
        i32x8 fo[FP];
        rest(I0);
        if constexpr (I0 == 0) {
#pragma unroll
            for (int j = 0; j < FT; ++j) sx[j] = *(const uint32_t*)(ls + st + 64 * j);
            sw = *(const uint32_t*)(lw + st);
#pragma unroll
            for (int j = 0; j < FT; ++j) {
                const i32x4 u = *(const i32x4*)(lb[0] + st + j * 16 * BK), v = *(const i32x4*)(lb[1] + st + j * 16 * BK);
                ft[j] = __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        }
#pragma unroll
        for (int i = 0; i < FP; ++i) {
            const i32x4 u = *(const i32x4*)(la[0] + st + (I0 + i) * 16 * BK), v = *(const i32x4*)(la[1] + st + (I0 + i) * 16 * BK);
            fo[i] = __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        read();
        f8_wait_lds();
        // float16 operands: the tokens' and the first row's here, a later row's under the instructions of the
        // one before it, which leaves the registers for tiles of 256 x 128
        f16x8 ho[EXACT ? 2 : 1][4], ht[EXACT ? FT : 1][4];
        auto half_row = [&](int i) {
#pragma unroll
            for (int h = 0; h < 4; ++h) ho[i & 1][h] = f8_half(fo[i][2 * h], fo[i][2 * h + 1]);
        };
        if constexpr (EXACT) {
            // waited for above: no use of them moves up
#pragma unroll
            for (int i = 0; i < FP; ++i) asm volatile("" : "+v"(fo[i]));
#pragma unroll
            for (int j = 0; j < FT; ++j) {
                asm volatile("" : "+v"(ft[j]));
#pragma unroll
                for (int h = 0; h < 4; ++h) ht[j][h] = f8_half(ft[j][2 * h], ft[j][2 * h + 1]);
            }
            half_row(0);
        }
        f8_barrier();
        __builtin_amdgcn_s_setprio(1);
        if constexpr (INSIDE) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                f32x4& r = acc[I0 + q / FT][q % FT];
                r = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fo[q / FT], ft[q % FT], r, 0, 0, 0, (int)sw, 0, (int)sx[q % FT]);
                during(q);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            if constexpr (I0 == 0) {
#pragma unroll
                for (int j = 0; j < FT; ++j)
                    s[j] = E8 ? f8_pow2(sx[j]) * f8_pow2(sw) : __builtin_bit_cast(float, sx[j]) * __builtin_bit_cast(float, sw);
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                f32x4& r = p[q % (AHEAD + 1)];
                r = (f32x4){0.f, 0.f, 0.f, 0.f};
                if constexpr (EXACT) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) r = __builtin_amdgcn_mfma_f32_16x16x32_f16(ho[(q / FT) & 1][h], ht[q % FT][h], r, 0, 0, 0);
                    if (q % FT == 0 && q / FT + 1 < FP) half_row(q / FT + 1);
                } else {
                    r = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fo[q / FT], ft[q % FT], r, 0, 0, 0, 0, 0, 0);
                }
                during(q);
                __builtin_amdgcn_sched_barrier(0);
                if (q >= AHEAD) add(I0, q - AHEAD, p[(q - AHEAD) % (AHEAD + 1)]);
            }
            if constexpr (!TWO)
#pragma unroll
                for (int q = Q - AHEAD; q < Q; ++q) add(I0, q, p[q % (AHEAD + 1)]);
            // the sums are added up here, and not where they are next used, behind a branch
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j) asm volatile("" : "+v"(acc[I0 + i][j]));
        }
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };
    using First = std::integral_constant<int, 0>;
    using Second = std::integral_constant<int, 1>;
    auto none = [](auto...) {};
    // Copies from .. to - 1 of stage `it`, spread over a part's matrix instructions: issued together they
    // hold up the waves for as long as their bytes take (8192^3 with scales of powers of two 357 us
    // against 419).  Where the multiply-adds fill that half step they go with the reads instead.
    auto together = [&](int it, int from, int to) {
#pragma unroll
        for (int j = from; j < to; ++j) copy(No{}, it, j);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto spread = [&](int it, int from, int to) {
        return [&copy, it, from, to](int q) {
#pragma unroll
            for (int j = from; j < to; ++j)
                if (q == (2 * (j - from) + 1) * Q / (2 * (to - from))) copy(No{}, it, j);
        };
    };
    // the same of a stage that may be partial, or not there
    auto spread_some = [&](int it, int from, int to) {
        return [&copy_some, it, from, to](int q) {
#pragma unroll
            for (int j = from; j < to; ++j)
                if (q == (2 * (j - from) + 1) * Q / (2 * (to - from))) copy_some(it, j, j + 1);
        };
    };
    // the first stages
    if constexpr (TWO) {
        copy_some(0, 0, L + 1);
        copy_some(1, 0, grp == 0 ? 5 : L + 1);
    } else {
        for (int q = 0; q < NST - 1; ++q) copy_some(q, 0, L + 1);
        if (INSIDE && (KG == 2 || grp == 1)) copy_some(NST - 1, 0, L + 1);
    }
#pragma unroll
    for (int i = 0; i < FO; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    if constexpr (!INSIDE) {
#pragma unroll
        for (int q = 0; q <= AHEAD; ++q) p[q] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < FT; ++j) s[j] = 0.f;
    }
    if constexpr (TWO) {
        // Quarter steps 4 s and 4 s + 2: the first group reads of stage s; 4 s + 1 and 4 s + 3: the
        // second.  X and the scales of stage s are read by quarter 4 s + 1, the codes of the first
        // parts by 4 s + 1, of the second by 4 s + 3.  Stage s + 2 takes their place:
        //   codes: copies 0 .. 3 and the scales' in quarter 4 s + 3, 4 .. 7 in 4 s + 5 (with the reads
        //   4 s + 2 and 4 s + 4); read from 4 s + 8 and 4 s + 10 on, so all but a wave's last 9 have
        //   landed when it waits, after its instructions;
        //   X: copies 0 .. 3 and the scales' in 4 s + 2, 4 .. 7 in 4 s + 4 (with the reads all in 4 s + 3);
        //   read from 4 s + 8 on: the wait, in the reads of 4 s + 7, leaves 5 (ahead of the copies: 0).
        static_assert(!TWO || (L == 8 && KG == 1 && BO == 256 && BT == 256), "two stages");
        if (nk > 1) {
            if (grp == 0) f8_wait_vm<5>();
            else f8_wait_vm<9>();
        } else {
            f8_wait_vm<0>();
        }
        f8_barrier();
        int it = 0;
        if (grp == 0) {
            for (; it + 2 < nfull; ++it) {
                if constexpr (INSIDE) step(First{}, it, none, spread(it + 1, 5, 9));
                else step(First{}, it, [&] { together(it + 1, 5, 9); }, none);
                f8_wait_vm<9>();
                f8_barrier();
                if constexpr (INSIDE) step(Second{}, it, none, spread(it + 2, 0, 5));
                else step(Second{}, it, [&] { together(it + 2, 0, 5); }, none);
                f8_wait_vm<9>();
                f8_barrier();
            }
            for (; it < nk; ++it) {
                step(First{}, it, [&] { copy_some(it + 1, 5, 9); }, none);
                f8_wait_vm<0>();
                f8_barrier();
                step(Second{}, it, [&] { copy_some(it + 2, 0, 5); }, none);
                f8_wait_vm<0>();
                f8_barrier();
            }
            f8_barrier();
        } else {
            f8_barrier();
            for (; it + 2 < nfull; ++it) {
                if constexpr (INSIDE) step(First{}, it, none, spread(it + 2, 0, 5));
                else step(First{}, it, none, none);
                f8_barrier();
                if constexpr (INSIDE) step(Second{}, it, [] { f8_wait_vm<5>(); }, spread(it + 2, 5, 9));
                else step(Second{}, it, [&] { f8_wait_vm<0>(); together(it + 2, 0, 9); }, none);
                f8_barrier();
            }
            for (; it < nk; ++it) {
                step(First{}, it, none, none);
                f8_barrier();
                step(Second{}, it, [&] { f8_wait_vm<0>(); copy_some(it + 2, 0, 9); }, none);
                f8_barrier();
            }
        }
    } else {
        // KG = 1: half steps 2 s (the first group reads stage s) and 2 s + 1 (the second does).  Under
        // its matrix instructions of stage s the first group copies stage s + NST - 1, in the place of
        // s - 1, the second s + NST, in the place of s; with the reads both copy s + NST - 1.  Stage s + 1
        // has landed before half step 2 s + 2: the first group waits at the end of 2 s + 1 (with the
        // reads: of 2 s), the second in its reads of stage s: NST - 2 stages may be in flight.
        // KG = 2: a group's own stages; under its instructions of stage s it copies s + NST and waits
        // after them.
        constexpr int FLY = (L + 1) * (KG == 2 && INSIDE ? NST - 1 : NST - 2);
        auto loop = [&](auto second) {
            constexpr bool G1 = decltype(second)::value && KG == 1;
            constexpr int DIST = INSIDE && (G1 || KG == 2) ? NST : NST - 1;
            int it = 0;
            for (; it + DIST < nfull; ++it) {
                if constexpr (INSIDE) {
                    step(First{}, it, [] { if (G1) f8_wait_vm<FLY>(); }, spread(it + DIST, 0, L + 1));
                    if (!G1) f8_wait_vm<FLY>();
                } else {
                    step(First{}, it, [&] { together(it + DIST, 0, L + 1); f8_wait_vm<FLY>(); }, none);
                }
                f8_barrier();
            }
            for (; it < nk; ++it) {
                if constexpr (INSIDE) {
                    step(First{}, it, [] { if (G1) f8_wait_vm<0>(); }, spread_some(it + DIST, 0, L + 1));
                    if (!G1) f8_wait_vm<0>();
                } else {
                    step(First{}, it, [&] { copy_some(it + DIST, 0, L + 1); f8_wait_vm<0>(); }, none);
                }
                f8_barrier();
            }
        };
        if (nk < NST) f8_wait_vm<0>();                    // stage 0 has landed
        else if (INSIDE && (KG == 2 || grp == 1)) f8_wait_vm<(L + 1) * (NST - 1)>();
        else f8_wait_vm<(L + 1) * (NST - 2)>();
        f8_barrier();
        if (KG == 2) {
            if (grp == 1) f8_barrier();
            loop(No{});
        } else if (grp == 0) {
            loop(No{});
        } else {
            f8_barrier();                                 // the second group runs half a step behind
            loop(Yes{});
        }
        if (KG == 2 && nk < nmax) {                       // the other group's last stage
            f8_barrier();
            f8_barrier();
        }
        if (grp == 0) f8_barrier();                       // every wave has read its last stage
    }
    rest(0);

    // KG = 2: group 0 finishes the first half of the wave's FO rows of fragments, group 1 the
    // second; each takes the other's sums of its half from LDS
    constexpr int FH = KG == 2 ? FO / 2 : FO;
    if constexpr (KG == 2) {
        f32x4* x = (f32x4*)smem + lane;                   // [group][wave][FH x FT][lane]
#pragma unroll
        for (int i = 0; i < FH; ++i)
#pragma unroll
            for (int j = 0; j < FT; ++j) {
                const f32x4 lo = acc[i][j], hi = acc[FH + i][j];
                f32x4 send, keep;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    send[e] = grp == 0 ? hi[e] : lo[e];
                    keep[e] = grp == 0 ? lo[e] : hi[e];
                }
                x[(((1 - grp) * 4 + wave) * (FH * FT) + i * FT + j) * 64] = send;
                acc[i][j] = keep;
            }
        f8_wait_lds();
        f8_barrier();
#pragma unroll
        for (int i = 0; i < FH; ++i)
#pragma unroll
            for (int j = 0; j < FT; ++j) acc[i][j] += x[((grp * 4 + wave) * (FH * FT) + i * FT + j) * 64];
    }
    const int64_t ob = o0 + wo * (BO / WO) + (KG == 2 ? grp * (FH * 16) : 0), tb = at.t0 + wt * (BT / WT) + r;
    const int64_t tend = at.end;
    bool bad[FT];
#pragma unroll
    for (int j = 0; j < FT; ++j) bad[j] = tb + 16 * j < tend && f8_bad(a, tb + 16 * j);
    bool stored = false;
    if constexpr (FH % 2 == 0) {
        if (a.splits == 1 && a.y_dtype != 0) {
            stored = true;
#pragma unroll
            for (int j = 0; j < FT; ++j)
#pragma unroll
                for (int i = 0; i < FH; i += 2)
                    f8_put_pair16(a, acc[i][j], acc[i + 1][j], tb + 16 * j, tend, ob + 16 * i, c, bad[j]);
        }
    }
    if (!stored) {
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int i = 0; i < FH; ++i) f8_out4(a, acc[i][j], tb + 16 * j, tend, ob + 16 * i + 4 * c, bad[j]);
    }
}

// HALF: a tile of 256 x 256 with no more than 128 rows, an expert's last, is one of 256 x 128 (PWQ_E4M3_SUMS,
// 16384 rows of 64 experts by 4096 x 4096 396 -> 379 us, of 128 by 1024 x 2048 103 -> 90; 32768 of 64, at the
// power limit, 622 -> 615).  It starts at another k than the full tiles of the same weights, so more of them
// comes from memory twice (32768 rows of 64 read 2447 MB in place of 1882).  One matrix has one such tile a
// column at most, and loses up to 1 % to it.
template <int BO, int BT, int NST, int WO, int KG, bool E8, bool EXACT, bool HALF>
__global__ __launch_bounds__(512) void f8_tile_kernel(F8Args a) {
    static_assert(!HALF || (BO == 256 && BT == 256), "half a tile");
    constexpr int MINE = f8_smem<BO, BT, NST, KG>, OTHER = HALF ? f8_smem<256, 128, 3, 1> : 0;
    __shared__ __attribute__((aligned(16))) uint8_t smem[MINE > OTHER ? MINE : OTHER];
    int to;
    F8Rows at{0, 0, 0};
    if (!f8_tile<BT>(a, blockIdx.x, to, at)) return;
    if constexpr (HALF) {
        if (at.end - at.t0 <= 128) {
            f8_tile_body<256, 128, 3, 4, 1, E8, EXACT>(a, smem, to, at);
            return;
        }
    }
    f8_tile_body<BO, BT, NST, WO, KG, E8, EXACT>(a, smem, to, at);
}

// ------------------------------------------------------------------ few tokens
// Few tokens, where the weights are the traffic or a launch's latency counts: a workgroup owns 16
// outputs by 16 tokens, its W waves share k in turns of U blocks each, every lane loads its
// fragments (16 bytes of one row) straight into registers, those of a turn while the turn before is
// multiplied, and the waves' sums meet in LDS.  No staging: a code is used once, and X comes from L2.
// The float16 instructions cost nothing here.  Loads past the rows or tokens take a 16-byte block of
// zeros as their address, so none waits behind a branch.  1 row by 8192 x 8192 17 us (4.0 TB/s), by 768 x
// 768 3.8 (an empty launch takes 2.2).  Rows of any alignment lose this way: 1 row by 28671 x 8191 108 us,
// 58 with the 64 x 32 tiles above.
template <int U, int W, bool E8>
__global__ __launch_bounds__(64 * W) void f8_row_kernel(F8Args a) {
    __shared__ f32x4 red[W][64];
    const F8Rows at = f8_rows<16>(a, blockIdx.z);
    if (at.t0 >= at.end) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, c = lane >> 4;
    const int64_t o0 = (int64_t)blockIdx.x * 16, t = at.t0 + r;
    const bool xin = t < at.end;
    const int64_t xt = f8_xrow(a, xin ? t : at.end - 1);
    const uint8_t* crow = a.C + ((int64_t)at.expert * a.m + (o0 + r < a.m ? o0 + r : a.m - 1)) * a.n + 16 * c;
    const uint8_t* xrow = a.X + (a.laid ? (xin ? t : at.end - 1) : xt) * a.ldx + 16 * c;
    const int64_t wat = f8_sw_at(a, at.expert, o0, 0);
    const bool bad = xin && f8_bad(a, t);
    struct Turn {
        i32x4 co[U][2], ct[U][2];
        float sx[U], sw[U];
    };
    Turn v[2];
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    const int64_t left_c = a.n - 16 * c;
    auto load = [&](Turn& q, int64_t b0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool bin = b0 + u < a.groups;
            const int64_t b = bin ? b0 + u : 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = (b0 + u) * F8_B + 64 * h;
                const bool in = k < left_c;
                q.co[u][h] = __builtin_nontemporal_load((const i32x4*)(in ? crow + k : (const uint8_t*)&f8_zeros));
                q.ct[u][h] = *(const i32x4*)(in && xin ? xrow + k : (const uint8_t*)&f8_zeros);
            }
            q.sx[u] = f8_get<E8>(a.sx, b * a.ldsx + xt);
            q.sw[u] = f8_get<E8>(a.sw, wat + b);
            if (!bin) q.sx[u] = q.sw[u] = 0.f;
        }
    };
    auto mult = [&](const Turn& q) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 4; ++h)
                p = __builtin_amdgcn_mfma_f32_16x16x32_f16(f8_half(q.co[u][h / 2][2 * (h & 1)], q.co[u][h / 2][2 * (h & 1) + 1]),
                                                           f8_half(q.ct[u][h / 2][2 * (h & 1)], q.ct[u][h / 2][2 * (h & 1) + 1]),
                                                           p, 0, 0, 0);
            const float s = q.sx[u] * q.sw[u];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(p[e], s, acc[e]);
        }
    };
    // turns of the whole workgroup, from a different one on each (see the tiles' order of k)
    constexpr int TURN = W * U;
    const int turns = (a.groups + TURN - 1) / TURN;
    int turn = (int)(blockIdx.x % (unsigned)turns);
    auto next = [&] {
        const int64_t b0 = (int64_t)turn * TURN + wave * U;
        turn = turn + 1 < turns ? turn + 1 : 0;
        return b0;
    };
    load(v[0], next());
    int left = turns;
    for (; left > 2; left -= 2) {
        load(v[1], next());
        mult(v[0]);
        load(v[0], next());
        mult(v[1]);
    }
    if (left == 2) {
        load(v[1], next());
        mult(v[0]);
        mult(v[1]);
    } else {
        mult(v[0]);
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) acc += red[w][lane];
    f8_out4(a, acc, t, at.end, o0 + 4 * c, bad);
}

// ------------------------------------------------------------------ splits
// The splits' sums of four outputs of a row at a time, in their order: a launch's latency, 4.5 us behind
// the tiles.  grid: x = outputs, y = rows
__global__ __launch_bounds__(256) void f8_join_kernel(F8Args a) {
    const int64_t o = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (o >= a.m) return;
    const int64_t size = a.T * a.m;
    int64_t t0 = 0, end = a.T;
    if (a.offsets) {
        t0 = a.offsets[0] < 0 ? 0 : a.offsets[0];
        end = a.offsets[a.experts] < a.T ? a.offsets[a.experts] : a.T;
    }
    for (int64_t t = t0 + blockIdx.y; t < end; t += gridDim.y) {
        const float* p = a.part + t * a.m + o;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        if (o + 4 <= a.m) {
            for (int k = 0; k < a.splits; ++k) {
                f32x4 v;
                __builtin_memcpy(&v, p + k * size, 16);
                s += v;
            }
        } else {
            for (int k = 0; k < a.splits; ++k)
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (o + e < a.m) s[e] += p[k * size + e];
        }
        f8_put4(a, s, t, o);
    }
}

// ------------------------------------------------------------------ copies
// X's row of each output row, and behind them the codes' rows, to rows of a multiple of 16 bytes with
// zeros at the end: 256 chunks of 16 bytes a wave at a time, four a lane.  The chunk that a row ends in
// is the row's last 16 bytes, moved down.  n >= 16, fewer than 2^30 chunks a row.  Memory's rate bounds
// it: 8000 + 1001 rows of 28671 in 88 us, 5.8 TB/s; with a wave to a row short rows took twice as long
// (64 x 2049 + 16000 rows of 1025: 104 us, now 50).
__global__ __launch_bounds__(256) void f8_lay_kernel(F8Args a, uint8_t* X, uint8_t* C) {
    const int64_t ld = f8_laid(a.n), chunks = (a.T + (int64_t)a.experts * a.m) * (ld / 16);
    const uint32_t cpr = (uint32_t)(ld / 16);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t at = ((int64_t)blockIdx.x * 4 + wave) * 256; at < chunks; at += (int64_t)gridDim.x * 1024) {
        const int64_t row0 = at / cpr;
        const uint32_t first = (uint32_t)(at - row0 * cpr);
        uint4 v[4];
        uint8_t* to[4];
        int drop[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t c = first + 64 * u + lane, down = c / cpr;
            const bool in = at + 64 * u + lane < chunks;
            const int64_t i = in ? row0 + down : 0, k = in ? 16 * (int64_t)(c - down * cpr) : 0;
            const int64_t past = k + 16 - a.n;
            drop[u] = past < 0 ? 0 : (int)past;
            const uint8_t* p = (i < a.T ? a.X + f8_xrow(a, i) * a.ldx : a.C + (i - a.T) * a.n) + (k - drop[u]);
            __builtin_memcpy(&v[u], p, 16);
            to[u] = in ? (i < a.T ? X + i * ld : C + (i - a.T) * ld) + k : nullptr;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (drop[u]) v[u] = f8_drop(v[u], drop[u]);
            if (to[u]) *(uint4*)to[u] = v[u];
        }
    }
}

// ------------------------------------------------------------------ launches
template <int BO, int BT, int NST, int WO, int KG, bool EXACT, bool HALF = false>
hipError_t f8_tile_go(F8Args a, bool e8, hipStream_t s) {
    a.tiles_m = (int)cdiv(a.m, BO);
    a.tiles_t = (int)f8_tiles_most(a.T, a.experts, BT);
    const dim3 grid((unsigned)(a.tiles_m * (int64_t)a.tiles_t), (unsigned)a.splits);
    if (e8) hipLaunchKernelGGL((f8_tile_kernel<BO, BT, NST, WO, KG, true, EXACT, HALF>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((f8_tile_kernel<BO, BT, NST, WO, KG, false, EXACT, HALF>), grid, dim3(512), 0, s, a);
    return hipGetLastError();
}

template <int U, int W>
hipError_t f8_row_go(F8Args a, bool e8, hipStream_t s) {
    a.tiles_t = (int)f8_tiles_most(a.T, a.experts, 16);
    const dim3 grid((unsigned)cdiv(a.m, 16), 1, (unsigned)a.tiles_t);
    if (e8) hipLaunchKernelGGL((f8_row_kernel<U, W, true>), grid, dim3(64 * W), 0, s, a);
    else hipLaunchKernelGGL((f8_row_kernel<U, W, false>), grid, dim3(64 * W), 0, s, a);
    return hipGetLastError();
}

template <int BO, int BT, int P, bool EXACT>
hipError_t f8_any_go(F8Args a, bool e8, hipStream_t s) {
    a.tiles_m = (int)cdiv(a.m, BO);
    a.tiles_t = (int)f8_tiles_most(a.T, a.experts, BT);
    const dim3 grid((unsigned)(a.tiles_m * (int64_t)a.tiles_t), (unsigned)a.splits);
    if (e8) hipLaunchKernelGGL((f8_any_kernel<BO, BT, P, true, EXACT>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((f8_any_kernel<BO, BT, P, false, EXACT>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t f8_run(F8Args a, bool e8, bool exact, const F8Plan& p, hipStream_t s) {
    a.splits = p.splits;
    a.kper = p.kper;
    hipError_t e;
    switch (p.kind) {
        case 0:
            e = a.offsets ? f8_tile_go<256, 256, 2, 2, 1, false, true>(a, e8, s) : f8_tile_go<256, 256, 2, 2, 1, false>(a, e8, s);
            break;
        case 1: e = exact ? f8_tile_go<256, 128, 3, 4, 1, true>(a, e8, s) : f8_tile_go<256, 128, 3, 4, 1, false>(a, e8, s); break;
        case 2: e = exact ? f8_tile_go<128, 128, 4, 2, 1, true>(a, e8, s) : f8_tile_go<128, 128, 4, 2, 1, false>(a, e8, s); break;
        case 3: e = exact ? f8_tile_go<128, 64, 4, 4, 1, true>(a, e8, s) : f8_tile_go<128, 64, 4, 4, 1, false>(a, e8, s); break;
        case 4: e = exact ? f8_tile_go<64, 64, 4, 2, 2, true>(a, e8, s) : f8_tile_go<64, 64, 4, 2, 2, false>(a, e8, s); break;
        case F8_ROW1: e = f8_row_go<2, 2>(a, e8, s); break;
        case F8_ROW2: e = f8_row_go<4, 4>(a, e8, s); break;
        case F8_ANY: e = exact ? f8_any_go<64, 32, 2, true>(a, e8, s) : f8_any_go<64, 32, 2, false>(a, e8, s); break;
        case F8_ANY + 1: e = exact ? f8_any_go<64, 64, 3, true>(a, e8, s) : f8_any_go<64, 64, 3, false>(a, e8, s); break;
        default: e = exact ? f8_any_go<128, 64, 3, true>(a, e8, s) : f8_any_go<128, 64, 3, false>(a, e8, s); break;
    }
    if (e != hipSuccess || a.splits == 1) return e;
    const dim3 grid((unsigned)cdiv(a.m, 1024), (unsigned)(a.T < 32768 ? a.T : 32768));
    hipLaunchKernelGGL(f8_join_kernel, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

bool f8_size_ok(int64_t T, int64_t m, int64_t experts) { return f8_plan_size_ok(T, m, experts); }
size_t f8_ws_bytes(int64_t T, int64_t n, int64_t m, int64_t experts) { return f8_plan_ws_bytes(T, n, m, experts); }

hipError_t f8_launch(const F8Call& c, hipStream_t s) {
    F8Args a{};
    a.X = c.X; a.sx = c.sx; a.C = c.C; a.sw = c.sw; a.offsets = c.offsets; a.rows = c.rows; a.Y = c.Y;
    a.part = (float*)c.ws; a.ldx = c.ldx; a.ldsx = c.ldsx; a.ldy = c.ldy; a.T = c.T; a.n = c.n; a.m = c.m;
    a.xrows = c.xrows; a.experts = (int)c.experts; a.groups = (int)cdiv(c.n, F8_B); a.y_dtype = c.y_dtype;
    // 32-bit offsets: from a tile's first row, or from X's with rows
    const bool near = c.n < ((int64_t)1 << 24) && (c.rows ? c.xrows * c.ldx < ((int64_t)1 << 32) : c.ldx < ((int64_t)1 << 24));
    const bool fast = c.n % 16 == 0 && c.ldx % 16 == 0 && aligned(c.X, 16) && aligned(c.C, 16) && near;
    const bool exact = !c.e4m3_sums;
    const F8Plan p = f8_plan(F8Shape{c.T, c.n, c.m, c.experts, exact, fast});
    if (p.lay) {
        uint8_t* const X = (uint8_t*)c.ws + f8_plan_ws_sums(p, c.T, c.m);
        uint8_t* const C = X + c.T * f8_laid(c.n);
        const int64_t blocks = cdiv((c.T + c.experts * c.m) * (f8_laid(c.n) / 16), 1024);
        hipLaunchKernelGGL(f8_lay_kernel, dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(256), 0, s, a, X, C);
        if (const hipError_t e = hipGetLastError()) return e;
        a.X = X; a.C = C; a.ldx = a.n = f8_laid(c.n); a.laid = true;
    }
    return f8_run(a, c.e8, exact, p, s);
}

}  // namespace pwq
