// f8_schedule.h -- how the block-scaled 8-bit-float products cut their work into
// pieces: arithmetic only, so that it also compiles for the host by itself.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define F8_HD __host__ __device__ __forceinline__
#else
#define F8_HD inline
#endif

namespace qk {
namespace f8 {

// See Schedule::plan.  One cost for both kernels, although a partial tile is 8 to
// 32 KB in f8_gemm.cu and 128 KB per CTA in f8_wide.cu.  Measured (us; a cost of 4,
// 16, 32, 64, never cut):
//   f8_gemm: 1 x 4096 x 14336 19.0 15.0 15.0 15.0 15.0; 4 x 9216 x 10000 23.7 23.7 23.7
//     22.8 22.8; 4 x 5120 x 19800 24.6 24.6 24.6 25.4 25.5; one row for each of 21 experts of
//     1024 x 2048 16.8 14.1 14.2 14.2 14.3; a layer of 4 tokens of 64 experts 43.2 37.1 37.0 37.0 37.0
//   f8_wide: 400 x 5120 x 5120 29.2 29.3 22.9 22.9 22.9; 512 x 17408 x 5120 54.1 54.2 54.2
//     54.1 61.5; 1100 x 17408 x 5120 105 106 105 105 119; 40 rows for each of 8 experts of 2560 x
//     9216 53.7 53.2 53.2 44.5 44.4, of 5 of 7936 x 5120 54.1 54.2 54.1 55.8 55.6
// Between 32 and 64 some shapes gain and some lose; 32 was taken.
constexpr int CUT_COST = 32;

F8_HD int smaller(int a, int b) { return a < b ? a : b; }
F8_HD int larger(int a, int b) { return a > b ? a : b; }
F8_HD int offset_at(const int32_t *offsets, int i) {
#ifdef __CUDA_ARCH__
    return __ldg(offsets + i);
#else
    return offsets[i];
#endif
}

// Tiles of `tokens` rows times nb row blocks of W for the group [lo, hi) of an
// expert, or -1 if the group is not taken: out of [0, R], or not behind every
// group before it (`top` is the largest offset up to and including lo).  Groups
// that are taken therefore have no row in common: no row of y is written by
// two experts, and there are at most R / tokens + E tiles times nb, which the
// caller has checked against 2^31.
F8_HD int group_tiles(int lo, int hi, int top, int R, int tokens, int nb) {
    if (lo < 0 || lo < top || hi < lo || hi > R) return -1;
    return (hi - lo + tokens - 1) / tokens * nb;
}

// A piece of a tile: tokens [row0, row0 + ntok) of expert e against block nblk
// of weight rows, K blocks [k0, k1).
struct Piece {
    int e, nblk, row0, ntok, k0, k1, tile;
};

// The pieces of this CTA (or pair) in order: first its share of the tiles that
// are cut along K, then its whole tiles.  (Tiles and K blocks of cut tiles are
// below 2^31: the caller checks the sizes.)
struct Schedule {
    const int *cum;  // shared memory: tiles before expert e, [E + 1]
    const int32_t *offsets;
    int E, R, kb, nb, G, c;
    int least;           // K blocks of cut tiles that a CTA has at least
    int step;            // tokens per tile; 0: the rows of an expert split evenly over its tiles
    int tiles, whole;    // tiles [0, whole) go round the CTAs uncut
    int units, sharing;  // K blocks of the cut tiles, and the CTAs that share them
    int u, u1;           // this CTA's of them, counted from tile `whole`
    int next_whole;

    // Which tiles are cut, and how.  Handing partial tiles over costs a CTA about
    // as much as CUT_COST K blocks, so
    // - tiles for half of the CTAs or fewer: each among G / tiles CTAs, nobody
    //   with parts of two tiles;
    // - else, when the last round would leave CTAs idle for longer than that: the
    //   tiles of the last round and of the full one before it (so that a cut tile
    //   has two or three parts) are shared out evenly over all CTAs;
    // - else none.
    F8_HD static void plan(int tiles, int kb, int G, int least, int &whole, int &units, int &sharing) {
        const int last = tiles % G;
        if (tiles <= G / 2) whole = 0;
        else if (last == 0 || static_cast<int64_t>(kb) * (G - last) <= static_cast<int64_t>(CUT_COST) * G) whole = tiles;
        else whole = tiles > G ? (tiles / G - 1) * G : 0;
        units = (tiles - whole) * kb;
        const int most = (kb + least - 1) / least;  // parts of a tile
        if (tiles <= G / 2) sharing = tiles * (G / larger(tiles, 1) < most ? G / larger(tiles, 1) : most);
        else sharing = G < units ? G : units;
    }
    F8_HD void init() {
        tiles = cum[E];
        plan(tiles, kb, G, least, whole, units, sharing);
        u = c < sharing ? static_cast<int>(static_cast<int64_t>(units) * c / sharing) : 0;
        u1 = c < sharing ? static_cast<int>(static_cast<int64_t>(units) * (c + 1) / sharing) : 0;
        next_whole = c;
    }
    F8_HD bool next(Piece &p) {
        if (u < u1) {
            const int t = u / kb;
            p.tile = whole + t;
            p.k0 = u - t * kb;
            p.k1 = smaller(kb, p.k0 + (u1 - u));
            u += p.k1 - p.k0;
        } else if (next_whole < whole) {
            p.tile = next_whole;
            next_whole += G;
            p.k0 = 0;
            p.k1 = kb;
        } else {
            return false;
        }
        int lo = 0, hi = E - 1;  // the expert whose tiles hold p.tile
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cum[mid] <= p.tile) lo = mid;
            else hi = mid - 1;
        }
        p.e = lo;
        const int local = p.tile - cum[lo];
        const int nt = (cum[lo + 1] - cum[lo]) / nb;
        const int r0 = offsets ? offset_at(offsets, lo) : 0;
        const int n = offsets ? offset_at(offsets, lo + 1) - r0 : R;
        // (an even share rounded up to 16 is at most a whole tile, so the last tile is not empty)
        const int per = step ? step : ((n + nt - 1) / nt + 15) & ~15;
        p.nblk = local / nt;
        const int tt = local - p.nblk * nt;
        p.row0 = r0 + tt * per;
        p.ntok = smaller(per, n - tt * per);
        return true;
    }
    // The CTAs [c0, c1] that hold a part of cut tile `tile`.
    F8_HD void sharers(int tile, int &c0, int &c1) const {
        const int64_t a = static_cast<int64_t>(tile - whole) * kb;
        c0 = static_cast<int>(((a + 1) * sharing - 1) / units);
        c1 = static_cast<int>(((a + kb) * sharing - 1) / units);
    }
};

}  // namespace f8
}  // namespace qk
