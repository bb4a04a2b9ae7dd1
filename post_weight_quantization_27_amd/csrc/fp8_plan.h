// Which kernel and how many splits of k a product of e4m3 codes takes (fp8_mm.hip): host code, no HIP,
// so that it can be compiled and checked alone.
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

namespace pwq {

inline int64_t f8_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t F8_STEP = 128;           // k of a block, and of a kernel's step
constexpr int64_t F8_SPLIT_MIN_K = 512;    // least k of a split

struct F8Plan {
    int kind;                      // one of the below, an index into f8_tiles, or F8_ANY + one into f8_any
    int splits;
    int64_t kper;
    double us = 0.0;               // estimate
    bool lay = false;              // the operands are copied to rows of 16-byte multiples first
};
constexpr int F8_ROW1 = -1, F8_ROW2 = -2, F8_ANY = 8;

// What decides: rows of Y, d_in, d_out, experts (1: one matrix), whether the sums are the float16
// instructions' (exact), whether operand rows start at multiples of 16 bytes and lie within 32-bit
// offsets of a tile's base (fast)
struct F8Shape {
    int64_t T, n, m, experts;
    bool exact, fast;
};

inline F8Plan f8_split(int kind, int64_t n, int64_t s) {
    const int64_t kper = f8_cdiv(f8_cdiv(n, s < 1 ? 1 : s), F8_STEP) * F8_STEP;
    return F8Plan{kind, (int)f8_cdiv(n, kper), kper};
}

// Tiles of bt rows: no more than these hold rows, whatever the experts' shares
inline int64_t f8_tiles_most(int64_t T, int64_t experts, int64_t bt) {
    if (experts <= 1) return f8_cdiv(T, bt);
    return T / bt + (T < experts ? T : experts);
}

// The kernels' side of the same (constexpr: device code too).  Offsets come from the device and may hold
// anything: what is counted stays within the `most` tiles of BT rows that were launched, which offsets that
// do not decrease never pass, so that 64 experts' tiles fit 31 bits and all tiles by outputs 24.
//
// an expert's rows lo .. hi - 1, taken into 0 .. T, in tiles of bt
constexpr int64_t f8_low(int64_t lo) { return lo < 0 ? 0 : lo; }
constexpr int64_t f8_high(int64_t hi, int64_t T) { return hi > T ? T : hi; }
constexpr int f8_own(int64_t lo, int64_t hi, int bt, int most) {
    const int64_t n = hi > lo ? (hi - lo + bt - 1) / bt : 0;
    return n < most ? (int)n : most;
}
// tiles of the experts before, `have`, and of 64 more
constexpr uint32_t f8_upto(uint32_t have, int more, int most) {
    return have + (uint32_t)more < (uint32_t)most ? have + (uint32_t)more : (uint32_t)most;
}
// Workgroup bid of tiles_t by tiles_m tiles: consecutive workgroups go to different XCDs, so each XCD takes
// a contiguous share of the tiles, in groups of up to 8 output tiles by all token tiles.
struct F8Place {
    int tt, to;                    // token tile, output tile
    bool there;
};
constexpr F8Place f8_place(uint32_t bid, uint32_t tiles_t, uint32_t tiles_m) {
    const uint32_t nt = tiles_t * tiles_m;
    if (bid >= nt) return F8Place{0, 0, false};
    const uint32_t x = bid & 7, per = nt >> 3, rem = nt & 7;
    const uint32_t id = x * per + (x < rem ? x : rem) + (bid >> 3);
    const uint32_t band = 8 * tiles_t, g = id / band, left = tiles_m - 8 * g;
    const uint32_t rows = left < 8 ? left : 8, in = id - g * band, down = in / rows;
    return F8Place{(int)down, (int)(8 * g + in - down * rows), true};
}

// What is expected of the experts' shares, which the host does not know: rows that choose any of them alike
struct F8Shares {
    double active, rows;           // experts that have rows, and how many each
};
inline F8Shares f8_shares(int64_t T, int64_t experts) {
    if (experts <= 1) return F8Shares{1.0, (double)T};
    const double a = (double)experts * -expm1((double)T * log1p(-1.0 / (double)experts));
    return F8Shares{a, (double)T / a};
}
// tiles of bt rows: one for each expert while its rows are few, or half of its last one empty
inline double f8_tiles_about(const F8Shares& e, int64_t T, int64_t experts, int64_t bt, double few) {
    if (experts <= 1) return (double)f8_cdiv(T, bt);
    return e.rows <= few ? e.active : (double)T / bt + 0.5 * e.active;
}

// Any alignment: the tile and the splits of k with the least estimate (us), rounds of tiles on 256
// compute units, of which workgroups that share one overlap a part.  Fitted to the times over 210 shapes
// with odd d_in (517 .. 14337 inputs, 769 .. 14337 outputs, 1 .. 3000 rows, one matrix and 7 or 32
// experts, float32 sums and the e4m3 instruction's): 1.2 % longer than the fastest in the geometric mean and
// 24 % at the worst; 64 x 64 tiles alone, unsplit, take 31 % longer in the mean.  333 rows by 5003 x 1601: 19.4
// us with 128 x 64, 21.9 with 64 x 64, 23.9 with 64 x 32; 16 by 4099 x 8191: 70, 52 and 35, with two splits of k
// 40, 32 and 23.
struct F8AnyCost {
    int bo, bt;
    float fixed, step, step_exact; // us per tile, and for each 128 k
};
constexpr F8AnyCost f8_any[] = {
    {64, 32, 0.3f, 0.323f, 0.362f},
    {64, 64, 1.07f, 0.473f, 0.585f},
    {128, 64, 2.26f, 0.755f, 0.989f},
};
inline F8Plan f8_plan_any(const F8Shape& s) {
    const F8Shares e = f8_shares(s.T, s.experts);
    const double mem = ((double)s.T * s.n + e.active * (double)s.m * s.n + 2.0 * s.T * s.m) * 1e-6 / 2.33;
    F8Plan best{F8_ANY, 1, s.n};
    double least = 1e30;
    for (int i = 0; i < (int)(sizeof(f8_any) / sizeof(f8_any[0])); ++i) {
        const F8AnyCost& c = f8_any[i];
        const double tiles = f8_tiles_about(e, s.T, s.experts, c.bt, c.bt / 2) * (double)f8_cdiv(s.m, c.bo);
        for (int64_t sp = 1; sp <= 8; sp *= 2) {
            if (sp > 1 && (s.n / sp < F8_SPLIT_MIN_K || tiles * sp > 2000.0)) break;
            const F8Plan p = f8_split(F8_ANY + i, s.n, sp);
            if (sp > 1 && p.splits < sp) continue;
            const double groups = tiles * p.splits / 256.0;
            const double rounds = s.experts > 1 ? (groups > 0.7 ? groups + 0.3 : 1.0) : ceil(groups);
            const double load = 0.175 * (groups > 1.0 ? groups : 1.0) + 0.825 * rounds;
            const double work = 4.2 + load * (c.fixed + (s.exact ? c.step_exact : c.step) * (double)f8_cdiv(p.kper, 128));
            double t = work > mem ? work + 0.05 * mem : mem + 0.05 * work;
            if (p.splits > 1) t += 3.4 + 0.28 * (double)p.splits * s.T * s.m * 4e-6;
            if (t < least) { least = t; best = p; }
        }
    }
    best.us = least;
    return best;
}

// What a tile costs on this chip: every compute unit holds one workgroup, which takes `fixed`
// microseconds and `step` more for each 128 k.
struct F8TileCost {
    int bo, bt;
    float fixed, step, step_exact; // us
};
constexpr F8TileCost f8_tiles[] = {
    {256, 256, 8.4f, 1.29f, 0.f},          // no float16 form: its fragments do not fit the registers
    {256, 128, 6.15f, 0.89f, 1.565f},
    {128, 128, 5.25f, 0.565f, 0.926f},
    {128, 64, 4.6f, 0.435f, 0.595f},
    {64, 64, 4.8f, 0.256f, 0.316f},
};
constexpr int F8_TILES = sizeof(f8_tiles) / sizeof(f8_tiles[0]);

// The least estimate (us) of: rounds of tiles on 256 compute units over 1 to 8 splits of k whose sums
// a second launch joins, and no less than memory takes; or the row kernel, whose workgroups stream their 16
// rows of codes once per 16 tokens.  The constants are fitted to the times of every kernel over 359 shapes,
// before experts' tiles of 256 x 256 had a half form.  Over 544 shapes of the kernels as they are (768 ..
// 28672 inputs and outputs, 1 .. 32768 rows, one matrix and 8 .. 128 experts) the choice takes 1.6 % longer than
// the fastest kernel in the geometric mean and 36 % at the worst (1024 rows of 8 experts by 2048 x 4096: 49
// against 36 us): of float32 sums 0.7 % for one matrix and 4.8 % for experts, of the e4m3 instruction's 1.1 %
// (powers of two 1.8) and 3.4 %.  128 x 128 tiles alone take 59 % longer in the mean and up to 5.3 times as long.
inline F8Plan f8_plan_fast(const F8Shape& s) {
    const F8Shares e = f8_shares(s.T, s.experts);
    const double bytes = ((double)s.T * s.n + e.active * (double)s.m * s.n + 2.0 * s.T * s.m) * 1e-6;      // MB
    const double mem = bytes / 5.66 + 4.76;
    F8Plan best{F8_ANY, 1, s.n};
    double least = 1e30;
    for (int i = 0; i < F8_TILES; ++i) {
        const F8TileCost& c = f8_tiles[i];
        const float step = s.exact ? c.step_exact : c.step;
        if (step == 0.f) continue;
        const double tiles = f8_tiles_about(e, s.T, s.experts, c.bt, c.bt / 2) * (double)f8_cdiv(s.m, c.bo);
        for (int64_t sp = 1; sp <= 8; sp *= 2) {
            if (sp > 1 && (s.n / sp < F8_SPLIT_MIN_K || tiles * sp > 1024.0)) break;
            const F8Plan p = f8_split(i, s.n, sp);
            if (sp > 1 && p.splits < sp) continue;
            const double groups = tiles * p.splits / 256.0;
            const double rounds = s.experts > 1 ? (groups > 0.6 ? groups + 0.4 : 1.0) : ceil(groups);
            const double work = 0.6 + rounds * (c.fixed + step * (double)p.kper / 128.0);
            double t = work > mem ? work + 0.1 * mem : mem + 0.1 * work;
            if (p.splits > 1) t += 3.4 + 0.335 * (double)p.splits * s.T * s.m * 4e-6;
            if (t < least) { least = t; best = p; }
        }
    }
    if (e.rows <= 256.0 && f8_tiles_most(s.T, s.experts, 16) <= 65535) {
        const double groups = (double)f8_cdiv(s.m, 16) * f8_tiles_about(e, s.T, s.experts, 16, 8.0) / 256.0;
        const double one = (1.0 + 0.31 * (e.rows < 16.0 ? e.rows : 16.0) / 16.0) * (groups > 1.0 ? groups : 1.0);
        // turns of 512 and of 2048 k, a last one that is not full counted half
        const int64_t turns1 = f8_cdiv(s.n, 512), turns2 = f8_cdiv(s.n, 2048);
        const double t1 = 2.8 + 0.79e-3 * 0.5 * (double)(s.n + 512 * turns1) * one + 0.38 * (double)turns1;
        const double t2 = 2.8 + 0.95e-3 * 0.5 * (double)(s.n + 2048 * turns2) * one + 0.17 * (double)turns2;
        if (t1 < least) { least = t1; best = f8_split(F8_ROW1, s.n, 1); }
        if (t2 < least) { least = t2; best = f8_split(F8_ROW2, s.n, 1); }
    }
    best.us = least;
    return best;
}

// d_in of the copies whose rows are multiples of 16 bytes
constexpr int64_t f8_laid(int64_t n) { return (n + 15) / 16 * 16; }

// The kernel of a call.  Rows of any length are copied to rows of 16-byte multiples first where that and
// the faster kernels are estimated to take less than the kernels for any alignment: a launch and the bytes
// at 6 TB/s.  8000 rows by 8191 x 8191, bfloat16: 931 us with 42 of copies, 2096 without; 700 by 4111 x
// 4099: 46 and 61; 333 by 5003 x 1601: 25 and 20.  With the e4m3 instruction's sums 496 and 1368, 38 and 49,
// 23 and 17, and over 90 shapes with odd d_in (32 .. 10000 rows) the choice takes 0.1 % longer than the better
// of the two in the mean and 6 % at the worst, no copies 11 % and up to 2.5 times as long.  A d_in that is a
// multiple of 16 is not copied, wherever its rows start: every call's workspace would have to hold the copies.
inline F8Plan f8_plan(const F8Shape& s) {
    if (s.fast) return f8_plan_fast(s);
    const F8Plan any = f8_plan_any(s);
    if (s.n % 16 == 0 || s.n < F8_STEP || s.n >= ((int64_t)1 << 24) - 16) return any;
    F8Shape l = s;
    l.n = f8_laid(s.n);
    F8Plan p = f8_plan_fast(l);
    p.us += 6.0 + 2e-6 * ((double)s.T + (double)s.experts * s.m) * (double)s.n / 6.0;
    p.lay = true;
    return p.us < any.us ? p : any;
}

inline bool f8_plan_size_ok(int64_t T, int64_t m, int64_t experts) {
    // work-items of a launch are counted in 32 bits: 512 for tiles of 64 x 64 at least
    return f8_tiles_most(T, experts, 64) * f8_cdiv(m, 64) < ((int64_t)1 << 23) && f8_cdiv(m, 16) < ((int64_t)1 << 23);
}

// The workspace: the splits' sums, and behind them the copies of X's rows and of the codes
inline size_t f8_plan_ws_sums(const F8Plan& p, int64_t T, int64_t m) {
    return p.splits > 1 ? ((size_t)p.splits * (size_t)T * (size_t)m * sizeof(float) + 15) / 16 * 16 : 0;
}
inline size_t f8_plan_ws_bytes(int64_t T, int64_t n, int64_t m, int64_t experts) {
    // whose sums, and where rows start, are the call's affair: room for any of its plans
    size_t most = 0;
    for (int i = 0; i < (n % 16 == 0 ? 4 : 2); ++i) {
        const F8Plan p = f8_plan(F8Shape{T, n, m, experts, (i & 1) != 0, (i & 2) != 0});
        const size_t copies = p.lay ? ((size_t)T + (size_t)experts * (size_t)m) * (size_t)f8_laid(n) : 0;
        const size_t b = f8_plan_ws_sums(p, T, m) + copies;
        most = b > most ? b : most;
    }
    return most;
}

}  // namespace pwq
