// latent_split.h -- how the work of absorbed latent attention is divided: whole
// numbers only, the same on the device and in a host program.
//
// The key tiles of all (sequence, unit of query rows) pairs are laid end to end and
// cut into equal ranges, one a worker (a CTA, or a pair of CTAs).  A unit that a cut
// falls into leaves partial sums, at most two a worker: in slot 2k if worker k does
// not hold its first tile, else in slot 2k + 1.
#pragma once

#ifdef __CUDACC__
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif

namespace pkv_split {

constexpr int TILE = 64;               // keys per tile

// How a kernel divides: (row, head) pairs of a unit, workers, and the numbers of
// sharers() and snap_of() below.
struct Rule {
    int unit, workers, each, few, snap;
};
// A pair of CTAs a worker (latent_decode.cu).  A tile costs a pair 1.4 us, a pair more
// the sequence 128 rows more to merge: three tiles at least, but up to 32 pairs with two,
// or one if that is all (one and a half would cut many units, each with its queries).
// (1,000 keys, 128 heads, one tile or two a pair: 15.8 and 17.2 us; eight sequences of
// 500 to 2,000, two or three: 29.4 and 26.0.  Their cuts left where they fall 26.4 us,
// moved 22.5.)
constexpr Rule PAIR = {128, 76, 3, 32, 3};
// A CTA a worker (latent_small.cu).  (16 sequences of 100 to 1,000 x 64 rows, one tile at
// least or two: 19.2 and 22.1 us; four of 2,000 to 5,000: 26.8 and 24.7.  256 of 50 to
// 300 x 16 rows, cuts left 32.1 us, moved 30.2.)
constexpr Rule ONE = {64, 152, 1, 0, 2};

PKV_HD int lesser(int a, int b) { return a < b ? a : b; }
PKV_HD int greater(int a, int b) { return a > b ? a : b; }

// A sequence as the kernels see it: first row, rows (0: none, or it was refused), keys.
struct Seq {
    int a, n, L;
};
PKV_HD int seq_tiles(const Seq &q) { return greater(1, (q.L + TILE - 1) / TILE); }
// tiles of all its units: every unit is charged the whole context (the causal
// end of a prompt chunk's earlier units leaves the rest of their charge empty)
PKV_HD int seq_cost(const Seq &q, int heads, int unit)
{
    if (q.n <= 0) return 0;
    return (int)((unsigned)(q.n * heads + unit - 1) / (unsigned)unit) * seq_tiles(q);
}

// Workers that W tiles are cut among: `each` tiles a worker at least, if there are as
// many; but up to `few` workers with one, if that is all, or two.
PKV_HD int sharers(int W, const Rule &r)
{
    return greater(1, lesser(r.workers, W <= r.few ? W : greater(W / r.each, lesser(W / 2, r.few))));
}
// The range of worker k of nc: W tiles in nc runs, the first W % nc one longer.
struct Cut {
    int each, extra;
    PKV_HD int begin(int k) const { return k * each + lesser(k, extra); }
    PKV_HD int owner(int pos) const
    {
        const bool longer = pos < extra * (each + 1);
        return (longer ? 0 : extra) + (pos - (longer ? 0 : extra * (each + 1))) / (longer ? each + 1 : each);
    }
};
PKV_HD Cut cut_of(int W, int nc) { return {W / nc, W - W / nc * nc}; }
// A cut that falls within this many tiles of a unit's end moves there: a worker
// would spend more on the few tiles' queries and partial sums.  (Less than a range,
// so that a worker loses no more than its own.)
PKV_HD int snap_of(const Cut &c, const Rule &r) { return lesser(r.snap, c.each * 2 / 3); }

// A place among all tiles, and within the sequence that holds it: unit and tile.
struct Place {
    int pos, u, t;
};
// The cut at `pos`, which lies in a sequence of KT tiles a unit that begins at b.
PKV_HD Place moved_cut(int pos, int b, int KT, int snap)
{
    const int u = (pos - b) / KT, t = pos - b - u * KT;
    if (t <= snap) return {pos - t, u, 0};
    if (KT - t <= snap) return {pos + KT - t, u + 1, 0};
    return {pos, u, t};
}

struct Item {
    Seq q;
    int s, r0, rows;     // the unit's first (row, head) pair within the sequence, and its pairs
    int j0, j1, kt;      // its tiles in this worker's range, and all its tiles
    int left;            // tiles of the range from its first one on
    PKV_HD bool whole() const { return j0 == 0 && j1 == kt; }
};
// Walks a worker's range; every role keeps one and sees the same items.  (No
// division but by constants and the head count: it runs between two items.)
struct Walk {
    int s, u, j, left;   // next: sequence, unit, tile; tiles left
};
// seq(s): sequence s
template <class SeqOf>
PKV_HD bool next_item(int num_seqs, int heads, int unit, Walk &w, Item &it, const SeqOf &seq)
{
    while (w.left > 0 && w.s < num_seqs) {
        const Seq q = seq(w.s);
        const int r0 = w.u * unit, all = q.n * heads;
        if (r0 >= all) {             // (a sequence without rows, too)
            ++w.s;
            w.u = w.j = 0;
            continue;
        }
        it.q = q;
        it.s = w.s;
        it.r0 = r0;
        it.rows = lesser(unit, all - r0);
        it.j0 = w.j;
        it.left = w.left;
        const int jend = lesser(seq_tiles(q), w.j + w.left);
        w.left -= jend - w.j;
        ++w.u;
        w.j = 0;
        const int last = q.n == 1 ? 0 : (int)((unsigned)(r0 + it.rows - 1) / (unsigned)heads);
        it.kt = greater(1, (q.L - q.n + last + 1 + TILE - 1) / TILE);       // tiles that its last row sees
        it.j1 = lesser(jend, it.kt);
        if (it.j0 < it.kt) return true;
    }
    return false;
}

// Partials of a unit whose first tiles, but not all, worker k of nc holds in a range
// that begins at `begin` and has `tiles`: they go up to the worker that holds the last
// tile that the unit's rows see (a cut in its last `snap` tiles has moved to its end).
PKV_HD int partials(const Cut &c, int nc, int snap, int begin, int tiles, const Item &it, int k)
{
    const int first = begin + (tiles - it.left);
    return greater(k, lesser(nc - 1, c.owner(first + lesser(it.kt, seq_tiles(it.q) - snap) - 1))) - k + 1;
}
// Where partial i of worker k's unit lies, and where worker k puts an item that is not whole.
PKV_HD int partial_slot(int k, int i) { return i == 0 ? 2 * k + 1 : 2 * (k + i); }
PKV_HD int own_slot(int k, const Item &it) { return 2 * k + (it.j0 == 0 ? 1 : 0); }

}  // namespace pkv_split
