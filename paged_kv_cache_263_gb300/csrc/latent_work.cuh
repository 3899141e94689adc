// latent_work.cuh -- what the two kernels of absorbed latent attention share: their
// parameters, how a worker finds its range (the division itself is latent_split.h),
// and their bounded waits.
#pragma once

#include "common.cuh"
#include "latent_split.h"

namespace {

__device__ uint32_t g_status;

using namespace pkv;
using pkv_split::Cut;
using pkv_split::Item;
using pkv_split::Seq;
using pkv_split::Walk;
using pkv_split::seq_tiles;

constexpr int TK = pkv_split::TILE;    // keys per tile
constexpr int MAX_WORKERS = pkv_split::ONE.workers;

struct LatentParams {
    uint16_t *out;
    const uint16_t *q;
    const int32_t *cu, *lens, *tables;
    int4 *desc;       // [workers] the unit to merge whose first tiles worker k holds: 1 (0: none), partials, rows, -
    int64_t *desc2;   // [workers] the unit's first (row, head)
    float *part_o;    // [2 workers][unit][512]
    float *part_ml;   // [2 workers][unit][2]
    int unit;         // (row, head) pairs of a unit, at most
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
__device__ __forceinline__ int seq_cost(const LatentParams &p, const Seq &q) { return pkv_split::seq_cost(q, p.heads, p.unit); }

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
    return pkv_split::next_item(p.num_seqs, p.heads, p.unit, w, it, [&](int s) -> Seq {
        const int i = s - g.s_first;
        return i < g.listed ? Seq{g.list[3 * i], g.list[3 * i + 1], g.list[3 * i + 2]} : read_seq(p, s, false);
    });
}

// Finds worker k's range (all threads of the CTA; two barriers and one more at the
// end): prefix sums of the sequences' costs, a run of consecutive sequences a
// thread.  scan: THREADS / 32 numbers, start: 3, cut: 4, list: 3 x listed, all in
// shared memory; start[0] = num_seqs, start[1] = start[2] = 0 beforehand.
template <int THREADS>
__device__ __forceinline__ Range find_range(const LatentParams &p, const pkv_split::Rule &rule, int k, bool flagging, int *scan,
                                            int *start, int *cut_sh, int *list, int listed)
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
    g.nc = pkv_split::sharers(W, rule);
    const Cut cut = pkv_split::cut_of(W, g.nc);
    g.snap = pkv_split::snap_of(cut, rule);
    const int w0 = k < g.nc ? cut.begin(k) : W, w1 = k < g.nc ? cut.begin(k + 1) : W;
    if (threadIdx.x == 0) {
        cut_sh[0] = cut.each;
        cut_sh[1] = cut.extra;
        if (w1 >= W) cut_sh[3] = W;
    }
    // where it begins and ends, by the thread whose sequences hold the place
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        const int pos = e == 0 ? w0 : w1;
        int b = before + incl - mine;
        if (w0 >= w1 || pos < b || pos >= b + mine) continue;
        int s = sa;
        for (; s < sb - 1; ++s) {
            const int cost = seq_cost(p, read_seq(p, s, false));
            if (pos < b + cost) break;
            b += cost;
        }
        const pkv_split::Place at = pkv_split::moved_cut(pos, b, seq_tiles(read_seq(p, s, false)), g.snap);
        cut_sh[2 + e] = at.pos;
        if (e == 0) {
            start[0] = s;
            start[1] = at.u;
            start[2] = at.t;
            // the first block ids, which the loads wait for
            asm volatile("prefetch.global.L1 [%0];" ::"l"(p.tables + (size_t)s * p.max_blocks + min(at.t * (TK / BS), p.max_blocks - 1)));
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

// What a worker that holds a unit's first tiles, but not all, writes into the merge list.
__device__ __forceinline__ void list_merge(const LatentParams &p, const Range &g, const Item &it, int k, int rows)
{
    const Cut cut = {g.cut[0], g.cut[1]};
    p.desc2[k] = (int64_t)it.q.a * p.heads + it.r0;
    p.desc[k] = make_int4(1, pkv_split::partials(cut, g.nc, g.snap, g.begin, g.tiles, it, k), rows, 0);
}

}  // namespace
