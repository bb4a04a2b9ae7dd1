// Which kernel and how many splits of k a product in 8-bit integers takes (w8a8.hip): host code, no
// HIP, so that it can be compiled and checked alone.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pwq {

inline int64_t w8_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int W8_SPLIT_MIN_K = 512;        // least k of a split of the tiles

struct W8Plan {
    int kind;                      // one of the below, or an index into w8_tiles
    int splits;
    int64_t kper;
};
constexpr int W8_ROW2 = -1, W8_ROW4 = -2, W8_ANY = 8;     // and W8_ANY + an index into w8_any

// k over `s` splits in whole steps of `step`
inline W8Plan w8_split(int kind, int64_t n, int64_t s, int64_t step) {
    const int64_t kper = w8_cdiv(w8_cdiv(n, s < 1 ? 1 : s), step) * step;
    return W8Plan{kind, (int)w8_cdiv(n, kper), kper};
}

// Any alignment: the tile and the splits of k with the least estimate (us), rounds of tiles as below,
// of which workgroups that share a compute unit overlap a part.  Fitted to the times over 289 shapes
// (100 .. 28670 inputs, most of them odd, 500 .. 28671 outputs, 1 .. 2000 tokens): 0.7 % longer
// than the fastest in the geometric mean and 19 % at the worst; 64 x 64 tiles alone, 128 x 128 from
// 1024 of those on, take 20 % longer in the mean.  In a loop over cold codes, float16 outputs: 333
// tokens by 5003 x 1601 13.7 us with 64 x 128, 16.6 with 64 x 64; 16 tokens by 28671 x 8191 58 with
// 128 x 32, 66 with 64 x 32, 83 with 64 x 64; 1 token by 4099 x 4095 13.0 with 64 x 32 in four
// splits, which the rule takes, 11.4 in two, 14.8 with 64 x 64 in one.
struct W8AnyCost {
    int bo, bt;
    float fixed, step;             // us per tile, and for each 128 k
};
constexpr W8AnyCost w8_any[] = {
    {64, 32, 0.55f, 0.29f}, {128, 32, 1.1f, 0.56f}, {64, 64, 1.1f, 0.42f}, {64, 128, 1.25f, 0.61f}, {128, 128, 2.7f, 1.05f},
};
inline W8Plan w8_plan_any(int64_t T, int64_t n, int64_t m) {
    const double mem = ((double)T * n + (double)m * n + 2.0 * T * m) * 1e-6 / 5.0 + 4.0;
    W8Plan best{W8_ANY, 1, n};
    double least = 1e30;
    for (int i = 0; i < (int)(sizeof(w8_any) / sizeof(w8_any[0])); ++i) {
        const W8AnyCost& c = w8_any[i];
        const int64_t tiles = w8_cdiv(T, c.bt) * w8_cdiv(m, c.bo);
        for (int64_t s = 1; s <= 8; s *= 2) {
            if (s > 1 && n / s < W8_SPLIT_MIN_K) break;
            const W8Plan p = w8_split(W8_ANY + i, n, s, 128);
            if (s > 1 && p.splits < s) continue;
            const double groups = (double)(tiles * p.splits) / 256.0, rounds = (double)w8_cdiv(tiles * p.splits, 256);
            const double load = 0.25 * (groups > 1.0 ? groups : 1.0) + 0.75 * rounds;
            double t = 3.3 + c.fixed * rounds + c.step * (double)w8_cdiv(p.kper, 128) * load;
            t = (t > mem ? t : mem) + 0.001 * t;
            if (p.splits > 1) t += 2.6 + 0.5 * (double)p.splits * T * m * 4e-6;
            if (t < least) { least = t; best = p; }
        }
    }
    return best;
}

// The tiles, and what one costs on this chip: every compute unit holds one workgroup, which takes
// `fixed` microseconds and `step` more for each 128 k.
struct W8TileCost {
    int bo, bt, bk;
    float fixed, step;
};
constexpr W8TileCost w8_tiles[] = {
    {256, 256, 64, 5.3f, 1.19f},
    {128, 256, 128, 3.3f, 0.64f},
    {128, 128, 128, 1.3f, 0.555f},
    {128, 64, 128, 0.55f, 0.48f},
    {64, 64, 128, 1.4f, 0.26f},
};
constexpr int W8_TILES = sizeof(w8_tiles) / sizeof(w8_tiles[0]);

// The least estimate (us) of: rounds of tiles on 256 compute units, each a fixed part and its steps
// of k, over 1 to 8 splits of k whose sums a second launch joins, and no less than memory takes;
// or the row kernel, whose workgroups stream their 16 rows of codes once per 16 tokens, at 19.5
// bytes per ns each.  The constants are fitted to the times of every kernel over some 600 shapes
// (512 .. 32000 inputs and outputs, 1 .. 4096 tokens): the choice takes 0.7 % longer than the
// fastest kernel in the geometric mean and 30 % at the worst (150 tokens by 4096 x 11008: 29.9
// against 23.0 us); 128 x 128 tiles alone take 58 % longer in the mean and up to 3.6 times as long.
inline W8Plan w8_plan_fast(int64_t T, int64_t n, int64_t m) {
    const double bytes = ((double)T * n + (double)m * n + 2.0 * T * m) * 1e-6;          // MB
    const double mem = bytes / 6.8 + 4.9;
    W8Plan best{0, 1, n};
    double least = 1e30;
    for (int i = 0; i < W8_TILES; ++i) {
        const W8TileCost& c = w8_tiles[i];
        const int64_t tiles = w8_cdiv(T, c.bt) * w8_cdiv(m, c.bo);
        for (int64_t s = 1; s <= 8; s *= 2) {
            if (s > 1 && n / s < W8_SPLIT_MIN_K) break;
            const W8Plan p = w8_split(i, n, s, c.bk);
            if (s > 1 && p.splits < s) continue;
            const double rounds = (double)w8_cdiv(tiles * p.splits, 256);
            const double work = 1.3 + rounds * (c.fixed + c.step * (double)p.kper / 128.0);
            double t = (work > mem ? work : mem) + 0.001 * work;
            if (p.splits > 1) t += 2.9 + 0.6 * (double)p.splits * T * m * 4e-6;
            if (t < least) { least = t; best = p; }
        }
    }
    if (T <= 1024) {
        const double groups = (double)w8_cdiv(w8_cdiv(m, 16) * w8_cdiv(T, 16), 256);
        const double one = 16e-3 * (double)n * (1.0 + 0.36 * (T < 16 ? T : 16) / 16.0) / 19.5;
        const double t = 1.9 + groups * one + 0.12 * (double)w8_cdiv(n, 1024);
        // turns of 8 waves x 128 k; of 256 k where they come out even on long rows (1 token by 8192 x
        // 8192: 14.7 against 15.8 us; 4096 x 8192 8.7 / 9.4; 4096 x 16384 13.8 / 23.2; 4096 x 14336
        // and 8192 x 10240 the same; 2048 x 8192 7.9 / 7.6; but 5120 x 5120 12.6 / 10.3)
        if (t < least) best = w8_split(n >= 8192 && n % 2048 == 0 ? W8_ROW4 : W8_ROW2, n, 1, 64);
    }
    return best;
}

// The kernel of a call; rows16: rows of X and codes start at multiples of 16 bytes
inline W8Plan w8_plan(int64_t T, int64_t n, int64_t m, bool rows16) {
    return rows16 ? w8_plan_fast(T, n, m) : w8_plan_any(T, n, m);
}

inline bool w8_plan_size_ok(int64_t T, int64_t m) {
    // work-items of a launch are counted in 32 bits: workgroups of 512 for tiles of 64 x 64 at least, of
    // 256 for 64 x 32
    return w8_cdiv(T, 64) * w8_cdiv(m, 64) < ((int64_t)1 << 23) && w8_cdiv(m, 16) < ((int64_t)1 << 23);
}

inline size_t w8_plan_ws_bytes(int64_t T, int64_t n, int64_t m) {
    // rows of 16-byte multiples or not is the pointers' affair, so there is room for either plan
    const W8Plan any = w8_plan_any(T, n, m);
    const W8Plan fast = n % 16 == 0 ? w8_plan_fast(T, n, m) : any;
    const int splits = any.splits > fast.splits ? any.splits : fast.splits;
    return splits > 1 ? (size_t)splits * (size_t)T * (size_t)m * sizeof(int32_t) : 0;
}

}  // namespace pwq
