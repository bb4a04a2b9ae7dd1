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
// The multiply runs on v_mfma_i32_16x16x64_i8 with C as the row operand (outputs) and X as the
// column operand (tokens): a lane holds 16 consecutive k of one row of each, in any order of k as
// long as both operands agree, and ends with four consecutive outputs of one token.  (The 32 x 32
// form does the same work per cycle but draws more power, which is what bounds large products:
// 8192^3 ran 9 % slower with it.)
#include "../../include/pwq.h"
#include "pwq_internal.h"
#include "pwq_common.h"
#include "w8a8_plan.h"

namespace pwq {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int W8_CUS = 256;                // compute units (a multiple of the 8 XCDs)

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

// What four outputs o .. o + 3, and a token, bring to the result.  Kernels load these before
// their first store: the compiler has to assume that a store may change them.
struct W8Quad {
    float w[4];
    int z[4];                      // 128 - zero
};
struct W8Tok {
    float s;
    int sum;
};

// Four outputs' values are read and written in one piece at any address; the last outputs of a
// row, where fewer than four are left, one by one.
__device__ __forceinline__ W8Quad w8_quad(const W8Args& a, int64_t o) {
    W8Quad q;
    uint16_t s[4], z[4] = {0, 0, 0, 0};
    if (o + 4 <= a.m) {
        __builtin_memcpy(s, a.sw + o, 8);
        if (a.zeros) __builtin_memcpy(z, a.zeros + o, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t i = o + e < a.m ? o + e : a.m - 1;
            s[e] = a.sw[i];
            if (a.zeros) z[e] = a.zeros[i];
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        q.w[e] = f16_bits_to_f32(s[e]);
        q.z[e] = 128 - (z[e] < 255 ? (int)z[e] : 255);
    }
    return q;
}
__device__ __forceinline__ W8Tok w8_tok(const W8Args& a, int64_t t) {
    t = t < a.T ? t : a.T - 1;
    return W8Tok{a.sx[t], a.zeros ? a.sums[t] : 0};
}

// Outputs o .. o + 3 of token t from their sums over k.  The scale of the row comes first (the sum
// times it stays inside float32's range), the token's last.
template <bool ZP>
__device__ __forceinline__ void w8_value4(float (&y)[4], i32x4 acc, const W8Quad& q, const W8Tok& k) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int s = ZP ? (int)((uint32_t)acc[e] + (uint32_t)q.z[e] * (uint32_t)k.sum) : acc[e];
        y[e] = ((float)s * q.w[e]) * k.s;
        asm("" : "+v"(y[e]));                             // rounded to float32 before the conversion, in every kernel
    }
}
__device__ __forceinline__ uint32_t w8_pair(const W8Args& a, float lo, float hi) {
    return a.y_dtype == 1 ? (uint32_t)f32_to_f16_bits(lo) | ((uint32_t)f32_to_f16_bits(hi) << 16)
                          : (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
}

template <bool ZP>
__device__ __forceinline__ void w8_put4(const W8Args& a, i32x4 acc, int64_t t, int64_t o, const W8Quad& q, const W8Tok& k) {
    float y[4];
    w8_value4<ZP>(y, acc, q, k);
    const int64_t i = t * a.ldy + o;
    if (a.y_dtype == 0) {
        float* p = (float*)a.Y + i;
        if (o + 4 <= a.m) {
            __builtin_memcpy(p, y, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (o + e < a.m) p[e] = y[e];
        }
    } else {
        uint16_t* p = (uint16_t*)a.Y + i;
        uint16_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a.y_dtype == 1 ? f32_to_f16_bits(y[e]) : f32_to_bf16_bits(y[e]);
        if (o + 4 <= a.m) {
            __builtin_memcpy(p, v, 8);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (o + e < a.m) p[e] = v[e];
        }
    }
}

// Two fragments' outputs in 16 bits, o0 .. o0 + 31 of the 16 tokens that a wave's lanes hold (lane
// row c: outputs 4 c .. 4 c + 3 of each fragment).  Two swaps between lane rows give row c the
// outputs 8 c .. 8 c + 7, so that a store writes 64 bytes of a row in one piece instead of 32.
template <bool ZP>
__device__ __forceinline__ void w8_put_pair16(const W8Args& a, i32x4 acc0, i32x4 acc1, int64_t t, int64_t o0, int c,
                                              const W8Quad& q0, const W8Quad& q1, const W8Tok& k) {
    float y0[4], y1[4];
    w8_value4<ZP>(y0, acc0, q0, k);
    w8_value4<ZP>(y1, acc1, q1, k);
    uint32_t even[2], odd[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto s = __builtin_amdgcn_permlane32_swap(w8_pair(a, y0[2 * h], y0[2 * h + 1]),
                                                        w8_pair(a, y1[2 * h], y1[2 * h + 1]), false, false);
        const auto r = __builtin_amdgcn_permlane16_swap(s[0], s[1], false, false);
        even[h] = r[0];
        odd[h] = r[1];
    }
    const uint32_t v[4] = {even[0], even[1], odd[0], odd[1]};
    const int64_t o = o0 + 8 * c;
    if (o >= a.m || t >= a.T) return;
    uint16_t* p = (uint16_t*)a.Y + t * a.ldy + o;
    if (o + 8 <= a.m) {
        __builtin_memcpy(p, v, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (o + e < a.m) p[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
    }
}

// Four outputs, or their sums over this split of k
template <bool ZP>
__device__ __forceinline__ void w8_out4(const W8Args& a, i32x4 acc, int64_t t, int64_t o, const W8Quad& q, const W8Tok& k) {
    if (o >= a.m || t >= a.T) return;
    if (a.splits > 1) {
        int32_t* p = a.part + ((int64_t)blockIdx.y * a.T + t) * a.m + o;
        if (o + 4 <= a.m) {
            __builtin_memcpy(p, &acc, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (o + e < a.m) p[e] = acc[e];
        }
        return;
    }
    w8_put4<ZP>(a, acc, t, o, q, k);
}

// ------------------------------------------------------------------ rows of 16-byte multiples
// BO x BT tile (outputs x tokens), eight waves, v_mfma_i32_16x16x64_i8 with the codes as the row
// operand, so that a lane ends with four consecutive outputs of one token.
//
// Operand rows go straight from memory into LDS (global_load_lds, 16 bytes a lane) in stages of
// BK k.  Row r of a stage keeps its 16-byte chunk c at a position xor-ed with a function of r
// chosen so that the 16 lanes which a 16-byte LDS read serves at a time (lanes 0-3, 12-15,
// 20-23, 24-27 of each half wave, and the rest) hit 16 different bank groups: the counters show
// no conflict.
//
// The waves work in two groups of four, one half step apart: while one group reads its fragments
// of a stage (and starts the copies of a later one), the other runs its MFMAs, with a barrier
// between the half steps.  Each SIMD holds one wave of each group, so its matrix unit always
// has the work of one of them.
//   KG = 1: both groups take every stage, each its half of the tile (WO x 8 / WO waves): the
//           least LDS traffic of the copies, for large tiles.
//   KG = 2: each group takes every other stage of k for the whole tile (WO x 4 / WO waves), with
//           stages of its own that its own waves copy; the two sums meet in LDS at the end.
//           The wave tiles are twice as large, which saves a third of the LDS reads on 64 x 64
//           tiles (48 tokens by 14336 x 4096: 14.3 against 15.3 us; 128 x 64 tiles are better off
//           with KG = 1 and a fourth stage: 64 tokens by 28672 x 8192 42 against 46 us, 2048 by
//           768 x 768 6.1 against 6.8, though 2048 by 1008 x 4096 16.0 against 14.5).
//
// Measured (kernel trace, operands cold): 8192^3 440-463 us, 8192 tokens by 28672 x 8192 1550-1640 us
// (2.3-2.5 POP/s).  The clock falls to 1.84 and 1.60 GHz there, which is what power leaves of 2.4, and
// the matrix units are busy 65 and 69 % of its cycles.  512 tokens by 8192 x 8192 41 us, 36 with the
// operands in the last cache (128 x 128 tiles, one per compute unit: 130 KB through LDS per 128 k
// are 1024 cycles at 128 bytes each, twice the multiplies', and the matrix units are busy 41 % of
// the time); 48 tokens by 28672 x 8192 43-45 us (5.3-5.6 TB/s of codes); one token by 8192 x 28672
// 41-43 us and 4.6 for the join (5.4-5.7 TB/s without it).  Between 17 and 512 tokens the tiles are
// far from both bounds: 64 by 8192 x 8192 28 us (the codes alone 11), 192 by 28672 x 8192 69 (41), 256
// by 17920 x 5120 46 (21), 320 by 28672 x 8192 98 (68): tiles padded with tokens that are not
// there, and too few of them for the chip.
// Stages of 64 k at KG = 2, which would fit 128 x 128 and 128 x 256 tiles, move 64-byte pieces of
// rows and take 30 % longer.
typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ const uint4 w8_zeros = {0u, 0u, 0u, 0u};

// s_waitcnt with only the vector-memory count constrained: vmcnt <= N
template <int N>
__device__ __forceinline__ void w8_wait_vm() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}
// all LDS reads of this wave have arrived
__device__ __forceinline__ void w8_wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }
// workgroup barrier without a fence: copies stay in flight across it
__device__ __forceinline__ void w8_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// position of chunk c in row r of a stage
template <int BK>
__device__ __forceinline__ int w8_pos(int r, int c) {
    static_assert(BK == 64 || BK == 128, "stage");
    return BK == 64 ? c ^ ((4 - (r >> 2)) & 3) : c ^ ((r >> 1) & 7);
}

// bid -> tile: consecutive workgroups go to different XCDs, so each XCD takes a contiguous share
// of the tiles, in groups of up to 8 output tiles by all token tiles
__device__ __forceinline__ void w8_map(const W8Args& a, int bid, int& to, int& tt) {
    const int nt = a.tiles_t * a.tiles_m;
    const int x = bid & 7, per = nt >> 3, rem = nt & 7;
    const int id = x * per + (x < rem ? x : rem) + (bid >> 3);
    const int g = id / (8 * a.tiles_t);
    const int rows = a.tiles_m - 8 * g < 8 ? a.tiles_m - 8 * g : 8;
    const int in = id - g * 8 * a.tiles_t;
    tt = in / rows;
    to = 8 * g + in - tt * rows;
}

// One workgroup per compute unit that goes through its tiles (3-4 % over a workgroup per tile on
// 8192 x 8192 x 2048 and 8192^3), where the registers allow it: with 256 x 256 tiles it gains
// nothing and the zero-point form spills.  (These keep the next tile's addresses beside this one's
// and spill 52 to 63 scalar registers into lanes of vector registers, none to memory.)
template <int BO, int BT, int KG>
constexpr bool w8_persist = KG == 1 && BO * BT < 65536;

template <int BO, int BT, int BK, int NST, int WO, int KG, bool ZP>
__global__ __launch_bounds__(512) void w8_tile_kernel(W8Args a) {
    constexpr int NW = 8 / KG, WT = NW / WO;              // waves that share a stage
    constexpr int FO = BO / WO / 16, FT = BT / WT / 16, KS = BK / 64;
    constexpr int ROWB = 1024 / BK;                       // rows per copy instruction of a wave
    constexpr int L = (BO + BT) / ROWB / NW;              // copies per wave and stage
    constexpr int ST = (BO + BT) * BK;
    constexpr bool PERSIST = w8_persist<BO, BT, KG>;
    static_assert(L * NW * ROWB == BO + BT && L * (NST - 2) < 64 && KG * NST * ST <= 163840, "tile");
    static_assert(KG == 1 || (FO % 2 == 0 && 8 * FO / 2 * FT * 1024 <= 2 * NST * ST), "the groups' sums fit the stages");
    __shared__ __attribute__((aligned(16))) uint8_t smem[KG * NST * ST];
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

    // copy j of this wave: ROWB rows from row q ROWB on, q = wave L + j, of the codes' BO rows
    // followed by the activations' BT; a lane brings the chunk that its position holds.  Rows
    // past the matrices repeat the last one (their outputs are not stored).
    const uint8_t* src[L];
    bool is_x[L];
    int chunk[L];
    int64_t o0, t0;
    // The order of k is free, so tiles that live on the codes' traffic start at different k:
    // where d_in is a multiple of 4096, rows that are read at the same k in step all come
    // from the same few memory channels (one token by 8192 x 28672 outputs: 52 us without, 44
    // with; at 8320 inputs 43 either way).  Large token tiles share X by k instead and start
    // together.
    constexpr int ROT = BT <= 128 ? 3 : 0;
    int rot;
    auto setup = [&](int tile) {
        int to, tt;
        w8_map(a, tile, to, tt);
        o0 = (int64_t)to * BO;
        t0 = (int64_t)tt * BT;
        rot = ROT && nfull > 0 ? (int)(((int64_t)to * ROT) % nfull) : 0;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int r = (wave * L + j) * ROWB + lane / (BK / 16);
            chunk[j] = w8_pos<BK>(r & 15, lane % (BK / 16));      // the xor undoes itself
            is_x[j] = (wave * L + j) * ROWB >= BO;
            if (is_x[j]) {
                const int64_t t = t0 + r - BO;
                src[j] = (const uint8_t*)a.X + (t < a.T ? t : a.T - 1) * a.ldx + kbeg + 16 * chunk[j];
            } else {
                const int64_t o = o0 + r;
                src[j] = a.C + (o < a.m ? o : a.m - 1) * a.n + kbeg + 16 * chunk[j];
            }
        }
    };
    auto copy = [&](int it) {
        uint8_t* S = lds + (it % NST) * ST + wave * (L * 1024);
        const int pos = it + rot;
        const int64_t k = (int64_t)(ROT && pos >= nfull ? pos - nfull : pos) * (KG * BK);
#pragma unroll
        for (int j = 0; j < L; ++j)
            __builtin_amdgcn_global_load_lds((const void*)(src[j] + k), (lds_ptr_t)(S + j * 1024), 16, 0, 0);
    };
    // the last stage where it ends past the rows: zeros for the activations, any bytes for the codes
    auto copy_end = [&](int it) {
        uint8_t* S = lds + (it % NST) * ST + wave * (L * 1024);
        const int64_t k = (int64_t)it * (KG * BK);
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const bool in = kbeg + k + 16 * chunk[j] < kend;
            const uint8_t* p = in ? src[j] + k : (is_x[j] ? (const uint8_t*)&w8_zeros : src[j] - 16 * chunk[j]);
            __builtin_amdgcn_global_load_lds((const void*)p, (lds_ptr_t)(S + j * 1024), 16, 0, 0);
        }
    };

    // the first NST - 1 stages of a tile
    auto begin = [&] {
#pragma unroll
        for (int q = 0; q < NST - 1; ++q) {
            if (q < nfull) copy(q);
            else if (q < nk) copy_end(q);
        }
    };

    i32x4 acc[FO][FT];
    const int r = lane & 15, c = lane >> 4;
    const uint8_t* la[KS];
    const uint8_t* lb[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const int o = r * BK + 16 * w8_pos<BK>(r, 4 * ks + c);
        la[ks] = lds + wo * (BO / WO) * BK + o;
        lb[ks] = lds + (BO + wt * (BT / WT)) * BK + o;
    }
    auto step = [&](int it, auto start_copy) {
        const int st = (it % NST) * ST;
        i32x4 fo[KS][FO], ft[KS][FT];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
            for (int j = 0; j < FT; ++j) ft[ks][j] = *(const i32x4*)(lb[ks] + st + j * 16 * BK);
#pragma unroll
            for (int i = 0; i < FO; ++i) fo[ks][i] = *(const i32x4*)(la[ks] + st + i * 16 * BK);
        }
        // stage it + NST - 1 takes the place of stage it - 1: the group ahead finished reading it
        // a step ago, the group behind before the barrier just passed.  This wave's copies of
        // stage it + 1 have landed before the barrier that lets the group ahead read it.
        start_copy();
        w8_wait_lds();
        if constexpr (ZP) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int i = 0; i < FO; ++i) {
                    // waited for above: the value passes through an empty asm so that no use of it moves up
                    asm volatile("" : "+v"(fo[ks][i]));
                    fo[ks][i] ^= (int)0x80808080;
                }
        }
        w8_barrier();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int i = 0; i < FO; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fo[ks][i], ft[ks][j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        w8_barrier();
    };
    int tile = blockIdx.x;
    setup(tile);
    begin();
    for (;;) {
#pragma unroll
        for (int i = 0; i < FO; ++i)
#pragma unroll
            for (int j = 0; j < FT; ++j) acc[i][j] = (i32x4){0, 0, 0, 0};
        if (nk >= NST - 1) w8_wait_vm<L * (NST - 2)>();
        else w8_wait_vm<0>();
        w8_barrier();
        if (grp == 1) w8_barrier();                           // the second group runs half a step behind
        int it = 0;
        for (; it + NST - 1 < nfull; ++it)
            step(it, [&] {
                copy(it + NST - 1);
                __builtin_amdgcn_sched_barrier(0);
                w8_wait_vm<L * (NST - 2)>();
            });
        for (; it < nk; ++it)
            step(it, [&] {
                if (it + NST - 1 < nk) copy_end(it + NST - 1);
                __builtin_amdgcn_sched_barrier(0);
                w8_wait_vm<0>();
            });
        if (KG == 2 && nk < nmax) {                           // the other group's last stage
            w8_barrier();
            w8_barrier();
        }
        if (grp == 0) w8_barrier();                           // every wave has read its last stage

        // KG = 2: group 0 finishes the first half of the wave's FO rows of fragments, group 1 the
        // second; each takes the other's sums of its half from LDS
        constexpr int FH = KG == 2 ? FO / 2 : FO;
        if constexpr (KG == 2) {
            i32x4* x = (i32x4*)smem + lane;                   // [group][wave][FH x FT][lane]
#pragma unroll
            for (int i = 0; i < FH; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j) {
                    const i32x4 lo = acc[i][j], hi = acc[FH + i][j];
                    i32x4 send, keep;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        send[e] = grp == 0 ? hi[e] : lo[e];
                        keep[e] = grp == 0 ? lo[e] : hi[e];
                    }
                    x[(((1 - grp) * 4 + wave) * (FH * FT) + i * FT + j) * 64] = send;
                    acc[i][j] = keep;
                }
            w8_wait_lds();
            w8_barrier();
#pragma unroll
            for (int i = 0; i < FH; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j) acc[i][j] += x[((grp * 4 + wave) * (FH * FT) + i * FT + j) * 64];
        }
        W8Quad q[FH];
        W8Tok tok[FT];
        const int64_t ob = o0 + wo * (BO / WO) + (KG == 2 ? grp * (FH * 16) : 0) + 4 * c, tb = t0 + wt * (BT / WT) + r;
#pragma unroll
        for (int i = 0; i < FH; ++i) q[i] = w8_quad(a, ob + 16 * i);
#pragma unroll
        for (int j = 0; j < FT; ++j) tok[j] = w8_tok(a, tb + 16 * j);
        // The next tile's first copies fly while this one's outputs are converted and stored
        tile += gridDim.x;
        const bool more = PERSIST && tile < a.tiles_t * a.tiles_m;
        if (more) {
            w8_wait_vm<0>();                                  // the scales just loaded, ahead of the copies
            setup(tile);
            begin();
        }
        bool stored = false;
        if constexpr (FH % 2 == 0) {
            if (a.splits == 1 && a.y_dtype != 0) {
                stored = true;
#pragma unroll
                for (int j = 0; j < FT; ++j)
#pragma unroll
                    for (int i = 0; i < FH; i += 2)
                        w8_put_pair16<ZP>(a, acc[i][j], acc[i + 1][j], tb + 16 * j, ob - 4 * c + 16 * i, c, q[i],
                                          q[i + 1], tok[j]);
            }
        }
        if (!stored) {
#pragma unroll
            for (int j = 0; j < FT; ++j)
#pragma unroll
                for (int i = 0; i < FH; ++i) w8_out4<ZP>(a, acc[i][j], tb + 16 * j, ob + 16 * i, q[i], tok[j]);
        }
        if (!more) break;
    }
}

// ------------------------------------------------------------------ any alignment
// BO x BT tile (outputs x tokens), four waves as 2 x 2, 128 k per step: rows may start at any byte
// and have any length.  Operands travel through registers into the same LDS layout as the tiles
// above, P steps ahead of their use; LDS has two buffers and a step one barrier.  No load stands
// behind a branch, so that the wait for one step's loads leaves the later steps' in flight.
//
// The last step may be partial: each 16 bytes past the end is the row's last 16 instead, moved
// down in registers, with 0 behind (X's zeros make the codes' bytes there irrelevant), fetched
// ahead like the others.
//
// 333 tokens by 5003 outputs in 16 bits, in a loop over cold codes: 9.8 us with rows of 1664 (whole
// cache lines; the tiles above), 12 with 1604 (a chunk of 128 takes two lines) and 14 with 1601 (16
// bytes from an odd address take the load path about twice as long, so tiles that read an operand
// less often gain); there with zero-points and float32 outputs 16.  Loads of the words around
// them, moved down by 0 to 3 bytes, were 1 to 5 % faster there and 10 % slower at few tokens, as
// they are five.  Long prompts are 2 to 3 times as long as on aligned rows (2000 tokens by 28671 x
// 8191: 1040 us; 2048 by 28672 x 8192: 460), more than copying both operands to aligned rows
// would cost; with 128 x 128 tiles the symmetric form needs 258 registers, two too many for a
// second workgroup on a compute unit, the zero-point form 248.

// The 16 bytes from byte `by` (0 .. 16) on, with 0 behind them
__device__ __forceinline__ uint4 w8_drop(uint4 v, int by) {
    if (by & 16) v = make_uint4(0u, 0u, 0u, 0u);
    if (by & 8) v = make_uint4(v.z, v.w, 0u, 0u);
    if (by & 4) v = make_uint4(v.y, v.z, v.w, 0u);
    const uint32_t b = (uint32_t)by & 3u;
    return make_uint4(__builtin_amdgcn_alignbyte(v.y, v.x, b), __builtin_amdgcn_alignbyte(v.z, v.y, b),
                      __builtin_amdgcn_alignbyte(v.w, v.z, b), __builtin_amdgcn_alignbyte(0u, v.w, b));
}

// 16 bytes of a row shorter than 16, from its byte k on, with 0 past its n
__device__ __forceinline__ uint4 w8_short(const uint8_t* row, int64_t k, int64_t n) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int e = 0; e < 16 && k + e < n; ++e) {
        const uint32_t byte = (uint32_t)row[k + e] << (8 * (e & 3));
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] |= c == e / 4 ? byte : 0u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int BO, int BT, int P, bool ZP>
__global__ __launch_bounds__(256) void w8_any_kernel(W8Args a) {
    constexpr int BK = 128, FO = BO / 32, FT = BT / 32;       // fragments of a wave
    constexpr int NC = (BO + BT) / 32;                        // chunks per thread
    constexpr int ST = (BO + BT) * BK;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * ST];
    int to, tt;
    w8_map(a, blockIdx.x, to, tt);
    const int64_t o0 = (int64_t)to * BO, t0 = (int64_t)tt * BT;
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
        if (r < BO) src[j] = a.C + (o0 + r < a.m ? o0 + r : a.m - 1) * a.n;
        else src[j] = (const uint8_t*)a.X + (t0 + r - BO < a.T ? t0 + r - BO : a.T - 1) * a.ldx;
        dst[j] = r * BK + 16 * w8_pos<BK>(r & 15, tid & 7);
    }
    const int nsteps = (int)cdiv(kend - kbeg, BK), nfull = (int)((kend - kbeg) / BK);
    auto at = [&](int it) {                                   // the step's k here, no later than the last 16 bytes
        const int64_t k = kbeg + (int64_t)(it < nsteps ? it : nsteps - 1) * BK + 16 * (tid & 7);
        return k < kend - 16 ? k : kend - 16;
    };
    auto fetch = [&](uint4 (&v)[NC], int it) {
        const int64_t k = at(it);
#pragma unroll
        for (int j = 0; j < NC; ++j) __builtin_memcpy(&v[j], src[j] + k, 16);
    };
    i32x4 acc[FO][FT];
#pragma unroll
    for (int i = 0; i < FO; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = (i32x4){0, 0, 0, 0};
    const int r = lane & 15, c = lane >> 4;
    auto multiply = [&](const uint8_t* S) {
        w8_wait_lds();
        w8_barrier();
#pragma unroll
        for (int ks = 0; ks < BK / 64; ++ks) {
            const int o = r * BK + 16 * w8_pos<BK>(r, 4 * ks + c);
            i32x4 fo[FO], ft[FT];
#pragma unroll
            for (int i = 0; i < FO; ++i) fo[i] = *(const i32x4*)(S + (wo * (BO / 2) + 16 * i) * BK + o);
#pragma unroll
            for (int j = 0; j < FT; ++j) ft[j] = *(const i32x4*)(S + (BO + wt * (BT / 2) + 16 * j) * BK + o);
#pragma unroll
            for (int i = 0; i < FO; ++i)
#pragma unroll
                for (int j = 0; j < FT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fo[i], ft[j], acc[i][j], 0, 0, 0);
        }
    };
    auto put = [&](uint8_t* S, int j, uint4 w) {
        if (ZP && j < BO / 32) { w.x ^= 0x80808080u; w.y ^= 0x80808080u; w.z ^= 0x80808080u; w.w ^= 0x80808080u; }
        *(uint4*)(S + dst[j]) = w;
    };
    // step `it` (a whole one: 128 k), whose chunks are in v; v is refilled for a later one under its
    // products
    auto step = [&](uint4 (&v)[NC], int it, int next) {
        uint8_t* S = lds + (it & 1) * ST;
#pragma unroll
        for (int j = 0; j < NC; ++j) put(S, j, v[j]);
        fetch(v, next);
        multiply(S);
    };
    auto last = [&](uint4 (&v)[NC], int it) {                 // one of the last, nothing to fetch
        uint8_t* S = lds + (it & 1) * ST;
        const int64_t drop = kbeg + (int64_t)it * BK + 16 * (tid & 7) - at(it);
#pragma unroll
        for (int j = 0; j < NC; ++j) put(S, j, it < nfull ? v[j] : w8_drop(v[j], (int)(drop < 16 ? drop : 16)));
        multiply(S);
    };
    if (a.n >= 16) {
        uint4 v[P][NC];
#pragma unroll
        for (int u = 0; u < P; ++u) fetch(v[u], u);
        int it = 0;
        for (; it + P <= nfull; it += P) {
#pragma unroll
            for (int u = 0; u < P; ++u) step(v[u], it + u, it + u + P);
        }
#pragma unroll
        for (int u = 0; u < P; ++u)
            if (it + u < nsteps) last(v[u], it + u);
    } else {                                                  // one step
#pragma unroll
        for (int j = 0; j < NC; ++j) put(lds, j, w8_short(src[j], 16 * (tid & 7), a.n));
        multiply(lds);
    }
    W8Quad q[FO];
    W8Tok tok[FT];
    const int64_t ob = o0 + wo * (BO / 2) + 4 * c, tb = t0 + wt * (BT / 2) + r;
#pragma unroll
    for (int i = 0; i < FO; ++i) q[i] = w8_quad(a, ob + 16 * i);
#pragma unroll
    for (int j = 0; j < FT; ++j) tok[j] = w8_tok(a, tb + 16 * j);
#pragma unroll
    for (int j = 0; j < FT; ++j)
#pragma unroll
        for (int i = 0; i < FO; ++i) w8_out4<ZP>(a, acc[i][j], tb + 16 * j, ob + 16 * i, q[i], tok[j]);
}

// ------------------------------------------------------------------ few tokens
// Few tokens by short rows, where a launch's latency counts, and one token, where the codes are the
// traffic: a workgroup owns 16 output rows by 16 tokens, its eight waves share k in turns of
// 64 U, every lane loads its fragments (16 bytes of one row) straight into registers, those of a
// turn while the turn before is multiplied, and the waves' sums meet in LDS.  No staging: a code
// is used once, and X comes from L2.  Loads past the rows or tokens take a 16-byte block of
// zeros as their address, so none waits behind a branch.  Measured (kernel trace, codes cold): one
// token by 768 x 768 3.4 us, by 8192 x 8192 16 us (4.2 TB/s; an empty launch takes 2.2).
template <int U, bool ZP>
__global__ __launch_bounds__(512) void w8_row_kernel(W8Args a) {
    __shared__ i32x4 red[8][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, c = lane >> 4;
    const int64_t o0 = (int64_t)blockIdx.x * 16, t = (int64_t)blockIdx.z * 16 + r;
    const uint8_t* crow = a.C + (o0 + r < a.m ? o0 + r : a.m - 1) * a.n;
    const bool xin = t < a.T;
    const uint8_t* xrow = (const uint8_t*)a.X + (xin ? t : 0) * a.ldx;
    const W8Quad q = w8_quad(a, o0 + 4 * c);              // ahead of the loop, for the end
    const W8Tok tok = w8_tok(a, t);
    i32x4 acc = {0, 0, 0, 0};
    i32x4 fo[2][U], ft[2][U];
    const int n = (int)a.n;
    auto load = [&](i32x4 (&co)[U], i32x4 (&ct)[U], int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + 64 * u + 16 * c;
            const bool in = k < n;
            co[u] = __builtin_nontemporal_load((const i32x4*)(crow + (in ? k : 0)));
            ct[u] = *(const i32x4*)(in && xin ? xrow + k : (const uint8_t*)&w8_zeros);
        }
    };
    auto mult = [&](i32x4 (&co)[U], i32x4 (&ct)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (ZP) co[u] ^= (int)0x80808080;
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(co[u], ct[u], acc, 0, 0, 0);
        }
    };
    // turns of the whole workgroup, from a different one on each (see the tiles' order of k)
    constexpr int TURN = 8 * 64 * U;
    const int turns = (n + TURN - 1) / TURN;
    int at = (int)(blockIdx.x % (unsigned)turns) * TURN + wave * (64 * U);
    auto next = [&] {
        const int k0 = at;
        at = at + TURN < turns * TURN ? at + TURN : wave * (64 * U);
        return k0;
    };
    load(fo[0], ft[0], next());
    int left = turns;
    for (; left > 2; left -= 2) {
        load(fo[1], ft[1], next());
        mult(fo[0], ft[0]);
        load(fo[0], ft[0], next());
        mult(fo[1], ft[1]);
    }
    if (left == 2) {
        load(fo[1], ft[1], next());
        mult(fo[0], ft[0]);
        mult(fo[1], ft[1]);
    } else {
        mult(fo[0], ft[0]);
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) acc += red[w][lane];
    w8_out4<ZP>(a, acc, t, o0 + 4 * c, q, tok);
}

// ------------------------------------------------------------------ splits
// The splits' sums of four outputs of a token at a time, scaled (one token, 8192 outputs: 4.6 us, a
// launch and two round trips to memory).  grid: x = outputs, y = tokens
template <bool ZP>
__global__ __launch_bounds__(256) void w8_join_kernel(W8Args a) {
    const int64_t o = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (o >= a.m) return;
    const W8Quad q = w8_quad(a, o);
    const int64_t size = a.T * a.m;
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        const W8Tok tok = w8_tok(a, t);
        const int32_t* p = a.part + t * a.m + o;
        i32x4 s = {0, 0, 0, 0};
        if (o + 4 <= a.m) {
            for (int k = 0; k < a.splits; ++k) {
                i32x4 v;
                __builtin_memcpy(&v, p + k * size, 16);
                s += v;
            }
        } else {
            for (int k = 0; k < a.splits; ++k)
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (o + e < a.m) s[e] += p[k * size + e];
        }
        w8_put4<ZP>(a, s, t, o, q, tok);
    }
}

// ------------------------------------------------------------------ launches
template <int BO, int BT, int BK, int NST, int WO, int KG>
hipError_t w8_tile_go(W8Args a, hipStream_t s) {
    a.tiles_m = (int)cdiv(a.m, BO);
    a.tiles_t = (int)cdiv(a.T, BT);
    const int64_t tiles = a.tiles_m * (int64_t)a.tiles_t;
    const dim3 grid((unsigned)(w8_persist<BO, BT, KG> && tiles > W8_CUS ? W8_CUS : tiles), (unsigned)a.splits);
    if (a.zeros) hipLaunchKernelGGL((w8_tile_kernel<BO, BT, BK, NST, WO, KG, true>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((w8_tile_kernel<BO, BT, BK, NST, WO, KG, false>), grid, dim3(512), 0, s, a);
    return hipGetLastError();
}

template <int U>
hipError_t w8_row_go(const W8Args& a, hipStream_t s) {
    const dim3 grid((unsigned)cdiv(a.m, 16), 1, (unsigned)cdiv(a.T, 16));
    if (a.zeros) hipLaunchKernelGGL((w8_row_kernel<U, true>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((w8_row_kernel<U, false>), grid, dim3(512), 0, s, a);
    return hipGetLastError();
}

template <int BO, int BT, int P>
hipError_t w8_any_go(W8Args a, hipStream_t s) {
    a.tiles_m = (int)cdiv(a.m, BO);
    a.tiles_t = (int)cdiv(a.T, BT);
    const dim3 grid((unsigned)(a.tiles_m * (int64_t)a.tiles_t), (unsigned)a.splits);
    if (a.zeros) hipLaunchKernelGGL((w8_any_kernel<BO, BT, P, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((w8_any_kernel<BO, BT, P, false>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t w8_run(W8Args a, const W8Plan& p, hipStream_t s) {
    a.splits = p.splits;
    a.kper = p.kper;
    hipError_t e;
    switch (p.kind) {
        case 0: e = w8_tile_go<256, 256, 64, 5, 4, 1>(a, s); break;
        case 1: e = w8_tile_go<128, 256, 128, 3, 2, 1>(a, s); break;
        case 2: e = w8_tile_go<128, 128, 128, 4, 2, 1>(a, s); break;
        case 3: e = w8_tile_go<128, 64, 128, 4, 4, 1>(a, s); break;
        case 4: e = w8_tile_go<64, 64, 128, 4, 2, 2>(a, s); break;
        case W8_ROW2: e = w8_row_go<2>(a, s); break;
        case W8_ROW4: e = w8_row_go<4>(a, s); break;
        case W8_ANY: e = w8_any_go<64, 32, 4>(a, s); break;
        case W8_ANY + 1: e = w8_any_go<128, 32, 4>(a, s); break;
        case W8_ANY + 2: e = w8_any_go<64, 64, 4>(a, s); break;
        case W8_ANY + 3: e = w8_any_go<64, 128, 3>(a, s); break;
        default: e = w8_any_go<128, 128, 2>(a, s); break;
    }
    if (e != hipSuccess || a.splits == 1) return e;
    const dim3 grid((unsigned)cdiv(a.m, 1024), (unsigned)(a.T < 32768 ? a.T : 32768));
    if (a.zeros) hipLaunchKernelGGL(w8_join_kernel<true>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(w8_join_kernel<false>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

bool w8_size_ok(int64_t T, int64_t m) { return w8_plan_size_ok(T, m); }
size_t w8_ws_bytes(int64_t T, int64_t n, int64_t m) { return w8_plan_ws_bytes(T, n, m); }

hipError_t w8_launch(const int8_t* X, int64_t T, int64_t n, int64_t ldx, const float* sx, const int32_t* sums,
                     const uint8_t* C, const uint16_t* sw, const uint16_t* zeros, int64_t m, void* Y, int y_dtype,
                     int64_t ldy, void* ws, hipStream_t s) {
    W8Args a{};
    a.X = X; a.sx = sx; a.sums = sums; a.C = C; a.sw = sw; a.zeros = zeros; a.Y = Y; a.part = (int32_t*)ws;
    a.ldx = ldx; a.ldy = ldy; a.T = T; a.n = n; a.m = m; a.y_dtype = y_dtype;
    const bool rows16 = n % 16 == 0 && ldx % 16 == 0 && aligned(X, 16) && aligned(C, 16);
    return w8_run(a, w8_plan(T, n, m, rows16), s);
}

}  // namespace pwq
