// latent_work.cuh -- what the two kernels of absorbed latent attention share: the
// division of a batch's work, and their bounded waits.
//
// The key tiles of all (sequence, unit of query rows) pairs are laid end to end and
// cut into equal ranges, one a worker (a CTA, or a pair of CTAs).  A unit that a cut
// falls into leaves fp32 partial sums, at most two a worker: in slot 2k if worker k
// does not hold its first tile, else in slot 2k + 1.
#pragma once

#include "common.cuh"

namespace {

__device__ uint32_t g_status;

using namespace pkv;

constexpr int TK = 64;                 // keys per tile
constexpr int MAX_WORKERS = 152;

struct LatentParams {
    uint16_t *out;
    const uint16_t *q;
    const int32_t *cu, *lens, *tables;
    int4 *desc;       // [workers] the unit to merge whose first tiles worker k holds: 1 (0: none), partials, rows, -
    int64_t *desc2;   // [workers] the unit's first (row, head)
    float *part_o;    // [2 workers][unit][512]
    float *part_ml;   // [2 workers][unit][2]
    int unit;         // (row, head) pairs of a unit, at most: 128 or 64
    int workers;
    int num_seqs, rows, heads, max_blocks, num_blocks;
    float scale_log2;
};

__device__ __forceinline__ void flag(uint32_t bits) { atomicOr(&g_status, bits); }

// PEER: what completes the phase comes from the other CTA of the cluster
template <bool PEER>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity)
{
    if (!PEER) return mbar_try_wait(bar, parity);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// bounded wait that also gives up once another warp of the CTA has
template <bool PEER = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    bool ok = try_wait<PEER>(bar, parity);
    if (!ok) {
        const unsigned long long t0 = globaltimer();
        for (uint32_t it = 1;; ++it) {
            if (try_wait<PEER>(bar, parity)) {
                ok = true;
                break;
            }
            if ((it & 63u) == 0) {
                if (*abort_flag) break;
                if (globaltimer() - t0 > WAIT_LIMIT_NS) {
                    *abort_flag = 1;
                    flag(ST_TIMEOUT);
                    break;
                }
            }
        }
    }
    return __all_sync(0xffffffffu, ok);   // the roles run warp-collective instructions: a warp leaves as a whole
}

// A sequence as the kernel sees it: n = 0 if it has no rows or was refused.
struct Seq {
    int a, n, L;
};
__device__ __forceinline__ Seq read_seq(const LatentParams &p, int s, bool flagging)
{
    Seq q;
    q.a = p.cu ? __ldg(p.cu + s) : s;
    const int b = p.cu ? __ldg(p.cu + s + 1) : s + 1;
    q.n = b - q.a;
    q.L = __ldg(p.lens + s);
    if (q.n == 0) return q;
    if (q.a < 0 || b < q.a || b > p.rows || q.L < 0 || q.L > p.max_blocks * BS || (q.L != 0 && q.L < q.n)) {
        if (flagging) flag(ST_BAD_LEN);
        q.n = 0;
    }
    return q;
}
__device__ __forceinline__ int seq_tiles(const Seq &q) { return max(1, (q.L + TK - 1) / TK); }
// tiles of all its units: every unit is charged the whole context (the causal
// end of a prompt chunk's earlier units leaves the rest of their charge empty)
__device__ __forceinline__ int seq_cost(const LatentParams &p, const Seq &q)
{
    if (q.n <= 0) return 0;
    return (int)((uint32_t)(q.n * p.heads + p.unit - 1) / (uint32_t)p.unit) * seq_tiles(q);
}

struct Item {
    Seq q;
    int s, r0, rows;     // the unit's first (row, head) pair within the sequence, and its pairs
    int j0, j1, kt;      // its tiles in this worker's range, and all its tiles
    int left;            // tiles of the range from its first one on
};
// Walks a worker's range; every role keeps one and sees the same items.  (No
// division and no memory but shared: it runs between two items of every role.)
struct Walk {
    int s, u, j, left;   // next: sequence, unit, tile; tiles left
};
// The range of worker k of nc: W tiles in nc runs, the first W % nc one longer.
struct Cut {
    int each, extra;
    __device__ __forceinline__ int begin(int k) const { return k * each + min(k, extra); }
    __device__ __forceinline__ int owner(int pos) const
    {
        const bool longer = pos < extra * (each + 1);
        return (longer ? 0 : extra) + (pos - (longer ? 0 : extra * (each + 1))) / (longer ? each + 1 : each);
    }
};

// A worker's range: where it starts, and how it was cut.
struct Range {
    Walk walk;
    int begin;               // its place among all tiles (which the host has made sure are fewer than 2^31)
    int tiles, nc, snap;     // its tiles; workers with work; tiles that a cut moves to a unit's end
    int s_first, listed;     // its first sequence; sequences tabled in shared memory from there on
    const int *list;
    const int *cut;          // shared memory: Cut's two numbers
};
__device__ __forceinline__ bool next_item(const LatentParams &p, const Range &g, Walk &w, Item &it)
{
    while (w.left > 0 && w.s < p.num_seqs) {
        const int i = w.s - g.s_first;
        Seq q;
        if (i < g.listed) q = {g.list[3 * i], g.list[3 * i + 1], g.list[3 * i + 2]};
        else q = read_seq(p, w.s, false);
        const int r0 = w.u * p.unit, all = q.n * p.heads;
        if (r0 >= all) {             // (a sequence without rows, too)
            ++w.s;
            w.u = w.j = 0;
            continue;
        }
        it.q = q;
        it.s = w.s;
        it.r0 = r0;
        it.rows = min(p.unit, all - r0);
        it.j0 = w.j;
        it.left = w.left;
        const int jend = min(seq_tiles(q), w.j + w.left);
        w.left -= jend - w.j;
        ++w.u;
        w.j = 0;
        const int last = q.n == 1 ? 0 : (int)((uint32_t)(r0 + it.rows - 1) / (uint32_t)p.heads);
        it.kt = max(1, (q.L - q.n + last + 1 + TK - 1) / TK);       // tiles that its last row sees
        it.j1 = min(jend, it.kt);
        if (it.j0 < it.kt) return true;
    }
    return false;
}

// Finds worker k's range (all threads of the CTA; two barriers and one more at the
// end): prefix sums of the sequences' costs, a run of consecutive sequences a
// thread.  EACH tiles a worker at least, if there are as many; but up to FEW workers
// with one, if that is all, or two.  A cut that falls within SNAP tiles of a unit's end moves there:
// the worker would spend more on the few tiles' queries and partial sums.  scan:
// THREADS / 32 numbers, start: 3, cut: 4, list: 3 x listed, all in shared memory;
// start[0] = num_seqs, start[1] = start[2] = 0 beforehand.
template <int THREADS, int EACH, int FEW, int SNAP>
__device__ __forceinline__ Range find_range(const LatentParams &p, int k, bool flagging, int *scan, int *start, int *cut_sh, int *list,
                                            int listed)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.num_seqs + THREADS - 1) / THREADS;
    const int sa = min(p.num_seqs, (int)threadIdx.x * per), sb = min(p.num_seqs, sa + per);
    int mine = 0;
    for (int s = sa; s < sb; ++s) mine += seq_cost(p, read_seq(p, s, flagging));
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int before = 0, W = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        const int t = scan[i];
        if (i < warp) before += t;
        W += t;
    }
    Range g;
    g.nc = max(1, min(p.workers, W <= FEW ? W : max(W / EACH, min(W / 2, FEW))));
    Cut cut;
    cut.each = W / g.nc;
    cut.extra = W - cut.each * g.nc;
    g.snap = min(SNAP, cut.each * 2 / 3);
    const int w0 = k < g.nc ? cut.begin(k) : W, w1 = k < g.nc ? cut.begin(k + 1) : W;
    if (threadIdx.x == 0) {
        cut_sh[0] = cut.each;
        cut_sh[1] = cut.extra;
        if (w1 >= W) cut_sh[3] = W;
    }
    // where it begins and ends, by the thread whose sequences hold the place
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        int pos = e == 0 ? w0 : w1, b = before + incl - mine;
        if (w0 >= w1 || pos < b || pos >= b + mine) continue;
        int s = sa;
        for (; s < sb - 1; ++s) {
            const int cost = seq_cost(p, read_seq(p, s, false));
            if (pos < b + cost) break;
            b += cost;
        }
        const int KT = seq_tiles(read_seq(p, s, false));
        int u = (pos - b) / KT, t = pos - b - u * KT;
        if (t <= g.snap) {
            pos -= t;
            t = 0;
        } else if (KT - t <= g.snap) {
            pos += KT - t;
            ++u;
            t = 0;
        }
        cut_sh[2 + e] = pos;
        if (e == 0) {
            start[0] = s;
            start[1] = u;
            start[2] = t;
            // the first block ids, which the loads wait for
            asm volatile("prefetch.global.L1 [%0];" ::"l"(p.tables + (size_t)s * p.max_blocks + min(t * (TK / BS), p.max_blocks - 1)));
        }
    }
    __syncthreads();
    g.s_first = start[0];
    for (int i = threadIdx.x; i < listed; i += THREADS) {
        const Seq q = g.s_first + i < p.num_seqs ? read_seq(p, g.s_first + i, false) : Seq{0, 0, 0};
        list[3 * i] = q.a;
        list[3 * i + 1] = q.n;
        list[3 * i + 2] = q.L;
    }
    g.begin = w0 < w1 ? cut_sh[2] : W;
    g.tiles = w0 < w1 ? max(0, cut_sh[3] - cut_sh[2]) : 0;
    g.walk = {g.s_first, start[1], start[2], g.tiles};
    g.listed = listed;
    g.list = list;
    g.cut = cut_sh;
    __syncthreads();
    return g;
}

// What a worker that holds a unit's first tiles, but not all, writes into the merge
// list: the partials go up to the worker that holds its last tile.
__device__ __forceinline__ void list_merge(const LatentParams &p, const Range &g, const Item &it, int k, int rows)
{
    const Cut cut = {g.cut[0], g.cut[1]};
    const int first = g.begin + (g.tiles - it.left);
    // (a cut in the unit's last `snap` tiles has moved to its end)
    const int kl = max(k, min(g.nc - 1, cut.owner(first + min(it.kt, seq_tiles(it.q) - g.snap) - 1)));
    p.desc2[k] = (int64_t)it.q.a * p.heads + it.r0;
    p.desc[k] = make_int4(1, kl - k + 1, rows, 0);
}

}  // namespace
