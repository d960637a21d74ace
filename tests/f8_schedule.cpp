// The schedule of the 8-bit-float products on the host, one CTA (or pair) after another: see test_f8_schedule.py.
#include "../mat_mul_gb300/csrc/f8_schedule.h"

using namespace qk::f8;

extern "C" {

// cum[0 .. E] and the number of groups that are refused.
int count_groups(const int32_t *offsets, int E, int R, int tokens, int nb, int *cum) {
    int bad = 0, top = 0;
    cum[0] = 0;
    for (int e = 0; e < E; ++e) {
        const int lo = offsets ? offsets[e] : 0;
        top = lo > top ? lo : top;
        int t = group_tiles(lo, offsets ? offsets[e + 1] : R, top, R, tokens, nb);
        if (t < 0) ++bad, t = 0;
        cum[e + 1] = cum[e] + t;
    }
    return bad;
}

// Every piece of every CTA, nine words each: CTA, expert, row block, first row, rows, first and last K block, tile, and
// the CTAs that share the tile as c0 * 65536 + c1 (-1: not cut).  Returns their number, or -1 if `room` is too small.
int walk(const int32_t *offsets, const int *cum, int E, int R, int nb, int kb, int step, int least, int G, int *out,
         int room, int *plan) {
    int n = 0;
    for (int c = 0; c < G; ++c) {
        Schedule s;
        s.cum = cum, s.offsets = offsets, s.E = E, s.R = R, s.nb = nb, s.kb = kb, s.step = step, s.least = least;
        s.G = G, s.c = c;
        s.init();
        plan[0] = s.tiles, plan[1] = s.whole, plan[2] = s.units, plan[3] = s.sharing;
        for (Piece p; s.next(p); ++n) {
            if (n == room) return -1;
            int cut = -1;
            if (p.k1 - p.k0 < kb) {
                int c0, c1;
                s.sharers(p.tile, c0, c1);
                cut = c0 * 65536 + c1;
            }
            const int row[9] = {c, p.e, p.nblk, p.row0, p.ntok, p.k0, p.k1, p.tile, cut};
            for (int i = 0; i < 9; ++i) out[9 * n + i] = row[i];
        }
    }
    return n;
}

int cut_cost() { return CUT_COST; }
}
