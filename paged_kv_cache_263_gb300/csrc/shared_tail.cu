// shared_tail.cu -- each sequence's own keys behind a prefix that a group shares, or
// whole contexts where no kernel of its own attends the prefixes (sm_103a).
//
// A work item is (sequence, set of its rows, part of its keys, KV head).  A set's rows x G
// heads, at most 16 columns, are attended as in the decode kernel: S^T[16 tokens][columns]
// = K Q^T and O^T[128][columns] += V^T P^T with mma.sync, one 16-token block a warp at a
// time, the softmax online (what is repaired in those products' loop belongs in the decode
// kernel's too, and the other way round).  What differs is how the work reaches the SM.  This kernel runs
// beside the one that attends the prefixes, on the few SMs that one leaves free, and
// an SM takes in at most 64 bytes a clock, 130 GB/s: so it must never stop loading.  A
// kernel with a CTA an item had its place in the batch, its block ids and its first
// loads to wait for at each start, and the join of its warps at each end: 3 us of 10
// for 32 blocks, 75 to 90 GB/s.
//  * Persistent CTAs, three an SM (two with 16 columns), of four (five) consumer warps
//    and a producer warp.  The producer finds the items, a CTA's next one through a counter
//    (or every grid-th one where all CTAs start together), and loads their queries and
//    blocks (one TMA box of 4 KiB for a K or V tile) into a ring for each consumer warp
//    that runs on across items: the next item's first blocks are there when the last
//    one's end.  (A ring of its own for each warp: a barrier's phases alternate between
//    two parities, so a warp has to see every phase of the stages that it waits for.)
//  * The next item is asked for when ASK_BLOCKS of the current one's blocks are left, not
//    at its start: an item that waits behind a long one could be another CTA's.  With items
//    of one part and one set, their sequence follows from their number; else the producer
//    walks over the batch, 32 sequences a step, 0.9 us each.  (Together: 48 sequences of 100
//    to 2,500 tokens beside two prefixes, fp8, 56.6 to 53.8 us for the call; 193 of one KV
//    head 30.3 to 26.9.  The counter for whole contexts too, where there are more items than
//    CTAs: 101 sequences of up to 12,356 tokens, fp8, 129 to 104.)
//  * The consumers' states are joined one after another through shared memory,
//    signalled by mbarriers, while warps that are done begin the next item.
//  * Results are partial ones, joined by the merge kernel, or the output itself.
#include "shared_prefix.h"
#include "tail_loads.h"
#include "trace.h"

#include <algorithm>

namespace {

__device__ uint32_t g_status;

using namespace pkv;

constexpr int QROW = 272;          // bytes of a column's query in shared memory: 256, kept off one bank
constexpr int SLOTS = 2;           // items ahead
constexpr int ASK_BLOCKS = 12;     // the next item is asked for when so many blocks of one are left to ask for

template <bool FP8, int NT>
struct TailLay {
    static constexpr int TILE = FP8 ? 2048 : 4096, STAGE = 2 * TILE;   // K and V of a block
    // an SM's CTAs and a CTA's consumer warps, as many as registers allow: 12 of 128
    // registers a thread, or 10 of 168
    static constexpr int CTAS = NT == 1 ? 3 : 2, CONSUMERS = NT == 1 ? 4 : 5;
    static constexpr int THREADS = 32 * (CONSUMERS + 1);
    static constexpr int RING = FP8 ? 4 : 2;                           // stages of a consumer warp
    static constexpr int STAGES = CONSUMERS * RING;
    static constexpr int COLS = 8 * NT;
    static constexpr int JOIN = COLS * (D + 2) * 4;                    // a warp's (O, max, sum)
    static constexpr int S_JOIN = STAGES * STAGE, S_Q = S_JOIN + JOIN;
    static constexpr int S_BAR = (S_Q + SLOTS * COLS * QROW + 15) / 16 * 16;
    static constexpr int SMEM = S_BAR + 512 + 1024;                    // (+ 1 KiB: aligned at run time)
    static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory of an SM");
    static_assert((2 * STAGES + 2 * SLOTS + CONSUMERS) * 8 + STAGES + SLOTS * 32 <= 512, "barrier area");
};

struct TailItem {
    int row0, n, L, g, b0, nb, slot, valid;   // L: keys from this kernel's key 0 on; slot: of the partial results
};

struct TailParams {
    SharedBatch b;
    __nv_bfloat16 *out16;            // the output, where one part is all there is; else null
    const uint16_t *q;
    const int32_t *block_tables;
    const float *k_scale, *v_scale;
    float *part_o, *part_ml;
    int *counter;                    // the next item, set by the kernel before; null: a CTA takes every grid-th
    int first;                       // ... and its first item is its own number
    int direct;                      // one part and one set of rows a sequence: its items are found without a walk
    int set_log2;                    // rows of a sequence in an item, a power of two
    int most;                        // items at most, of a batch that keeps the rules
    int hq, hkv, group, num_blocks, part_blocks, fine_from, fine_blocks, part_stride, part_off;
    int whole;                       // contexts from their first key on, the prefix through the group's first row
    int beside;                      // launched to run beside the kernel before, whose inputs were complete too
    float scale_log2;
};

__device__ __forceinline__ void flag(uint32_t bits) { atomicOr(&g_status, bits); }

__device__ __forceinline__ void tma_box_3d(uint32_t dst, const CUtensorMap *map, int32_t y, uint32_t bar, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %2}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar), "l"(pol)
        : "memory");
}
__device__ __forceinline__ void tma_box_2d(uint32_t dst, const CUtensorMap *map, int32_t y, uint32_t bar, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar), "l"(pol)
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// 32 sequences at a time, as the producer walks over the batch: their items lie end to
// end in the order (sequence, part, KV head), the last fastest
struct TailWindow {
    int w0, base, total;             // first sequence, items before it, items in it
    int incl, ns, sets;              // this lane's sequence: items up to it, parts, sets of rows
    SharedSeq q;
};
__device__ __forceinline__ void load_window(const TailParams &p, TailWindow &w, int lane)
{
    const int s = w.w0 + lane;
    w.q = shared_seq_window(p.b, w.w0, lane);
    w.ns = w.sets = 0;
    if (s < p.b.num_seqs) {
        if (w.q.state == SEQ_BAD) flag(ST_BAD_LEN);
        if (w.q.state == SEQ_OK && w.q.n > 0) {
            const int blocks = (w.q.L - (p.whole ? 0 : w.q.P) + BS - 1) / BS;
            const int part = s < p.fine_from ? p.part_blocks : p.fine_blocks;
            w.ns = (blocks + part - 1) / part;
            w.sets = (w.q.n + (1 << p.set_log2) - 1) >> p.set_log2;
        }
    }
    w.incl = w.ns * p.hkv * w.sets;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, w.incl, o);
        if (lane >= o) w.incl += t;
    }
    w.total = __shfl_sync(0xffffffffu, w.incl, 31);
    // rows of sequences without a context, where no merge kernel writes them (this CTA goes
    // through all windows; else the CTAs that come upon them do)
    if (p.out16 && !p.direct && blockIdx.x == 0)
        zero_rows(p.out16, p.hq, s < p.b.num_seqs && w.q.state == SEQ_EMPTY, w.q.row0, w.q.n, lane);
}

template <bool FP8, int NT>
__global__ void __launch_bounds__(TailLay<FP8, NT>::THREADS, TailLay<FP8, NT>::CTAS)
    shared_tail_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ TailParams p)
{
    using LY = TailLay<FP8, NT>;
    constexpr int STAGES = LY::STAGES, CONSUMERS = LY::CONSUMERS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    // barriers: a stage's block landed / was used; an item and its queries are there /
    // were read; warp w's state is in the join buffer (w > 0) / warp 0 has read it (w = 0)
    const uint32_t b_full = sbase + LY::S_BAR, b_free = b_full + 8 * STAGES, b_item = b_free + 8 * STAGES,
                   b_taken = b_item + 8 * SLOTS, b_join = b_taken + 8 * SLOTS;
    TailItem *items = reinterpret_cast<TailItem *>(smem + LY::S_BAR + (2 * STAGES + 2 * SLOTS + CONSUMERS) * 8);
    volatile uint8_t *stage_ok = reinterpret_cast<volatile uint8_t *>(items + SLOTS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_free + 8 * i, 1);
        }
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(b_item + 8 * i, 1);
            mbar_init(b_taken + 8 * i, CONSUMERS);
        }
        for (int i = 0; i < CONSUMERS; ++i) mbar_init(b_join + 8 * i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (!p.beside) griddep_wait();
    // (a wait that runs out ends its warp; the others' waits on it run out in turn)
    auto wait = [&](uint32_t bar, int phase) -> bool {
        const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, phase & 1));
        if (!ok && lane == 0) flag(ST_TIMEOUT);
        return ok;
    };

    if (warp == CONSUMERS) {
        // ======================= producer
        uint64_t pol;
        if (p.whole) asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
        else asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
        int u = 0, k = 0;        // blocks handed to this lane's consumer warp, and items
        int asked = 0;           // items whose queries were asked for
        bool ok = true;
        // (in lane 0; its answer is waited for where it is used)
        auto ask = [&](int idx) -> int {
            return !p.counter ? idx + (int)gridDim.x : lane == 0 ? atomicAdd(p.counter, 1) : 0;
        };
        int idx = p.first ? (int)blockIdx.x : ask(0);
        // (direct: the window of the item that is likely to be its first)
        TailWindow w = {};
        if (p.direct) w.w0 = min((int)blockIdx.x / p.hkv, p.b.num_seqs - 1) & ~31;
        load_window(p, w, lane);
        idx = __shfl_sync(0xffffffffu, idx, 0);
        for (;; ++k) {
            int at = 32, part = 0, r = 0;    // the item's sequence in the window (32: no more), its head and set
            if (p.direct) {
                // sequence and head from the number; sequences with nothing to attend are passed over
                for (; idx < p.b.num_seqs * p.hkv; idx = __shfl_sync(0xffffffffu, ask(idx), 0)) {
                    const int in = idx / p.hkv;
                    r = idx - in * p.hkv;
                    if ((in & ~31) != w.w0) {
                        w.w0 = in & ~31;
                        load_window(p, w, lane);
                    }
                    if (__shfl_sync(0xffffffffu, w.ns, in & 31)) {
                        at = in & 31;
                        break;
                    }
                    const int n = __shfl_sync(0xffffffffu, w.q.state == SEQ_EMPTY ? w.q.n : 0, in & 31);
                    const int row0 = __shfl_sync(0xffffffffu, w.q.row0, in & 31), width = p.group * (D / 8);
                    if (p.out16)
                        for (int i = lane; i < n * width; i += 32)
                            reinterpret_cast<uint4 *>(p.out16 + ((size_t)(row0 + i / width) * p.hq + r * p.group) * D)[i % width] =
                                make_uint4(0u, 0u, 0u, 0u);
                }
            } else {
                while (idx - w.base >= w.total && w.w0 + 32 < p.b.num_seqs && w.base + w.total <= p.most) {
                    w.base += w.total;
                    w.w0 += 32;
                    load_window(p, w, lane);
                }
                const int x = idx - w.base;
                if (x < w.total) {
                    at = __ffs(__ballot_sync(0xffffffffu, w.incl > x)) - 1;
                    const int of = p.hkv * __shfl_sync(0xffffffffu, w.sets, at);
                    r = x - (__shfl_sync(0xffffffffu, w.incl, at) - __shfl_sync(0xffffffffu, w.ns, at) * of);
                    part = r / of;
                    r -= part * of;
                }
            }
            TailItem it = {};
            int s = 0, P = 0, first = 0;
            if (at < 32) {
                s = w.w0 + at;
                P = __shfl_sync(0xffffffffu, w.q.P, at);
                first = __shfl_sync(0xffffffffu, w.q.first, at);
                // (the rows of set i of a sequence begin at i << set_log2, and their keys end where
                // those of the last one do; the parts are those of the whole sequence)
                const int n = __shfl_sync(0xffffffffu, w.q.n, at), sets = __shfl_sync(0xffffffffu, w.sets, at);
                it.g = sets == 1 ? r : r / sets;
                const int i0 = (r - it.g * sets) << p.set_log2, keys = __shfl_sync(0xffffffffu, w.q.L, at) - (p.whole ? 0 : P);
                it.row0 = __shfl_sync(0xffffffffu, w.q.row0, at) + i0;
                it.n = min(1 << p.set_log2, n - i0);
                it.L = keys - n + i0 + it.n;
                const int part_blocks = s < p.fine_from ? p.part_blocks : p.fine_blocks;
                it.b0 = part * part_blocks;
                it.nb = min((keys + BS - 1) / BS, it.b0 + part_blocks) - it.b0;
                it.slot = p.part_off + part;
                it.valid = 1;
            }
            const int sl = k % SLOTS;
            if (k >= SLOTS && !(ok = wait(b_taken + 8 * sl, k / SLOTS - 1))) break;
            const int cols = it.n * p.group;
            if (lane == 0) {
                items[sl] = it;
                mbar_arrive_expect_tx(b_item + 8 * sl, it.valid ? cols * 256 : 0);
            }
            __syncwarp();
            if (!it.valid) break;
            asked = k + 1;
            fence_proxy_async_smem();
            if (lane < cols)
                bulk_load(sbase + LY::S_Q + (sl * LY::COLS + lane) * QROW,
                          p.q + ((size_t)(it.row0 + lane / p.group) * p.hq + it.g * p.group + lane % p.group) * D, 256,
                          b_item + 8 * sl);
            // block j of the part: the prefix's through the group's first row (whole), the
            // others through the sequence's own
            const int pb = P / BS;
            const int32_t *own = p.block_tables + (size_t)s * p.b.max_blocks + (p.whole ? 0 : pb) + it.b0;
            const int32_t *shared = p.block_tables + (size_t)first * p.b.max_blocks + it.b0;
            const int from_shared = p.whole ? pb - it.b0 : 0;
            auto load_ids = [&](int j) -> int { return j < it.nb ? (j < from_shared ? shared : own)[j] : -1; };
            // a block for each consumer warp at a time, from the lane of the warp's number
            int next = 0;
            bool asked_next = false;
            int ids = load_ids(lane), ahead = load_ids(32 + lane), base = 0;   // ids of blocks base + lane, base + 32 + lane
            for (int j0 = 0; j0 < it.nb; j0 += CONSUMERS) {
                // (late: an item that waits behind a long one could be another CTA's)
                if (!asked_next && it.nb - j0 <= ASK_BLOCKS) {
                    next = ask(idx);
                    asked_next = true;
                }
                if (j0 - base >= 32) {
                    base += 32;
                    ids = ahead;
                    ahead = load_ids(base + 32 + lane);
                }
                const int at = j0 + lane - base;
                const int id0 = __shfl_sync(0xffffffffu, ids, at & 31), id1 = __shfl_sync(0xffffffffu, ahead, at & 31);
                const int id = at < 32 ? id0 : id1;
                const bool mine = lane < CONSUMERS && j0 + lane < it.nb;
                const int st = lane * LY::RING + u % LY::RING;
                bool there = true;
                if (mine && u >= LY::RING) there = mbar_wait_bounded(b_free + 8 * st, (u / LY::RING - 1) & 1);
                ok = __all_sync(0xffffffffu, there);
                if (!ok) {
                    if (lane == 0) flag(ST_TIMEOUT);
                    break;
                }
                if (mine) {
                    const uint32_t bar = b_full + 8 * st, dst = sbase + st * LY::STAGE;
                    const bool in = id >= 0 && id < p.num_blocks;
                    stage_ok[st] = in;
                    if (in) {
                        const int y = (id * p.hkv + it.g) * BS;
                        fence_proxy_async_smem();
                        mbar_arrive_expect_tx(bar, LY::STAGE);
                        if constexpr (FP8) {
                            tma_box_2d(dst, &kmap, y, bar, pol);
                            tma_box_2d(dst + LY::TILE, &vmap, y, bar, pol);
                        } else {
                            tma_box_3d(dst, &kmap, y, bar, pol);
                            tma_box_3d(dst + LY::TILE, &vmap, y, bar, pol);
                        }
                    } else {
                        flag(ST_BAD_BLOCK);
                        mbar_arrive(bar);        // completes the phase without data
                    }
                    ++u;
                }
                __syncwarp();
            }
            if (!ok) break;
            idx = __shfl_sync(0xffffffffu, next, 0);
        }
        griddep_launch_dependents();
        // (this lane's consumer warp's blocks, and the items' queries)
        pkv_tail::drain(
            lane < CONSUMERS ? u : 0, LY::RING, asked, SLOTS, ok,
            [&](int i) { (void)mbar_wait_bounded(b_full + 8 * (lane * LY::RING + i % LY::RING), (i / LY::RING) & 1); },
            [&](int i) { (void)mbar_wait_bounded(b_item + 8 * (i % SLOTS), (i / SLOTS) & 1); });
        __syncwarp();
        // the grid completes after the kernel it ran beside: what waits for it sees both
        if (p.beside && blockIdx.x == 0) griddep_wait();
        return;
    }

    // ======================= consumers
    const int gq = lane >> 2, cq = lane & 3;
    int u = 0;                   // blocks that this warp has been through
    for (int k = 0;; ++k) {
        const int sl = k % SLOTS;
        if (!wait(b_item + 8 * sl, k / SLOTS)) return;
        const TailItem it = items[sl];
        if (!it.valid) return;
        const int cols = it.n * p.group;
        // ---- Q fragments (B operand of S^T = K . Q^T)
        uint32_t qf[NT][8][2];
        int lim[NT][2];          // keys that this lane's two columns of each n-tile see
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int c = nt * 8 + gq;
            const uint32_t qa = sbase + LY::S_Q + (sl * LY::COLS + c) * QROW;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t x0, x1;
                if constexpr (!FP8) {
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x0) : "r"(qa + 32 * kk + 4 * cq));
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x1) : "r"(qa + 32 * kk + 4 * cq + 16));
                } else {
                    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(x0), "=r"(x1) : "r"(qa + 32 * kk + 8 * cq));
                    x0 = pack_f16(bf16_lo(x0), bf16_hi(x0));
                    x1 = pack_f16(bf16_lo(x1), bf16_hi(x1));
                }
                qf[nt][kk][0] = c < cols ? x0 : 0u;
                qf[nt][kk][1] = c < cols ? x1 : 0u;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = (nt * 8 + 2 * cq + e) / p.group;     // row of the column
                lim[nt][e] = i < it.n ? it.L - it.n + i + 1 : it.L;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b_taken + 8 * sl);
        float sl2 = p.scale_log2, vsc = 1.f;
        if constexpr (FP8) {
            sl2 *= p.k_scale[it.g];
            vsc = p.v_scale[it.g];
        }
        float o[NT][8][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
        }
        for (int j = warp; j < it.nb; j += CONSUMERS) {
            const int st = warp * LY::RING + u % LY::RING;
            if (!wait(b_full + 8 * st, u / LY::RING)) return;
            ++u;
            const int t0 = (it.b0 + j) * BS, nvalid = min(BS, it.L - t0);
            const uint32_t kb = sbase + st * LY::STAGE, vb = kb + LY::TILE;
            if (stage_ok[st]) {
                // ---------------- S^T = K . Q^T
                float sacc[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sacc[nt][i] = 0.f;
                const int mi = lane >> 3, ktok = ((mi & 1) << 3) | (lane & 7);
                if constexpr (!FP8) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const int chunk = 2 * kk + (mi >> 1);
                        uint32_t a0, a1, a2, a3;
                        ldsm_x4(kb + (chunk >> 3) * 2048 + ktok * 128 + (((chunk & 7) ^ (ktok & 7)) << 4), a0, a1, a2, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_bf16(sacc[nt], a0, a1, a2, a3, qf[nt][kk][0], qf[nt][kk][1]);
                    }
                } else {
#pragma unroll
                    for (int i2 = 0; i2 < 4; ++i2) {
                        const int chunk = 2 * i2 + (mi >> 1);
                        uint32_t r0, r1, r2, r3;
                        ldsm_x4(kb + ktok * 128 + ((chunk ^ (ktok & 7)) << 4), r0, r1, r2, r3);
                        // (the order of the dims inside a step is permuted, and the queries' with it)
                        const uint32_t a0 = e4m3x2_to_f16x2(r0 & 0xffff), a2 = e4m3x2_to_f16x2(r0 >> 16);
                        const uint32_t a1 = e4m3x2_to_f16x2(r1 & 0xffff), a3 = e4m3x2_to_f16x2(r1 >> 16);
                        const uint32_t c0 = e4m3x2_to_f16x2(r2 & 0xffff), c2 = e4m3x2_to_f16x2(r2 >> 16);
                        const uint32_t c1 = e4m3x2_to_f16x2(r3 & 0xffff), c3 = e4m3x2_to_f16x2(r3 >> 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(sacc[nt], a0, a1, a2, a3, qf[nt][2 * i2][0], qf[nt][2 * i2][1]);
                            mma_f16(sacc[nt], c0, c1, c2, c3, qf[nt][2 * i2 + 1][0], qf[nt][2 * i2 + 1][1]);
                        }
                    }
                }
                // ---------------- online softmax (log2 domain), per column
                uint32_t pb[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = t0 + gq + ((i >> 1) << 3) < lim[nt][i & 1] ? sacc[nt][i] * sl2 : -INFINITY;
                    float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) {
                        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
                        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
                    }
                    const float mn0 = fmaxf(m[nt][0], mx0), mn1 = fmaxf(m[nt][1], mx1);
                    // (no key seen yet: exponents against 0, so that p = 0)
                    const float r0 = mn0 == -INFINITY ? 0.f : mn0, r1 = mn1 == -INFINITY ? 0.f : mn1;
                    const float al0 = ex2(m[nt][0] - r0), al1 = ex2(m[nt][1] - r1);
                    m[nt][0] = mn0;
                    m[nt][1] = mn1;
                    const float p0 = ex2(x[0] - r0), p1 = ex2(x[1] - r1), p2 = ex2(x[2] - r0), p3 = ex2(x[3] - r1);
                    l[nt][0] = l[nt][0] * al0 + (p0 + p2);
                    l[nt][1] = l[nt][1] * al1 + (p1 + p3);
                    if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
                        for (int jj = 0; jj < 8; ++jj) {
                            o[nt][jj][0] *= al0;
                            o[nt][jj][1] *= al1;
                            o[nt][jj][2] *= al0;
                            o[nt][jj][3] *= al1;
                        }
                    }
                    pb[nt][0] = movmatrix_t(FP8 ? pack_f16(p0, p1) : pack_bf16(p0, p1));
                    pb[nt][1] = movmatrix_t(FP8 ? pack_f16(p2, p3) : pack_bf16(p2, p3));
                }
                // ---------------- O^T += V^T . P^T  (values past the last key count as zeros)
                if constexpr (!FP8) {
                    const int vtok = ((mi >> 1) << 3) | (lane & 7);
                    const uint32_t m01 = (2 * cq < nvalid ? 0x0000ffffu : 0u) | (2 * cq + 1 < nvalid ? 0xffff0000u : 0u);
                    const uint32_t m23 = (2 * cq + 8 < nvalid ? 0x0000ffffu : 0u) | (2 * cq + 9 < nvalid ? 0xffff0000u : 0u);
#pragma unroll
                    for (int jj = 0; jj < 8; ++jj) {
                        const int chunk = 2 * jj + (mi & 1);
                        uint32_t a0, a1, a2, a3;
                        ldsm_x4_t(vb + (chunk >> 3) * 2048 + vtok * 128 + (((chunk & 7) ^ (vtok & 7)) << 4), a0, a1, a2, a3);
                        if (nvalid < BS) {
                            a0 &= m01;
                            a1 &= m01;
                            a2 &= m23;
                            a3 &= m23;
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_bf16(o[nt][jj], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    }
                } else {
                    uint32_t w[4][4];  // tokens 2c, 2c+1, 2c+8, 2c+9; 16 bytes of chunk gq each
#pragma unroll
                    for (int ti = 0; ti < 4; ++ti) {
                        const int tok = 2 * cq + (ti & 1) + ((ti >> 1) << 3);
                        lds128(vb + tok * 128 + ((gq ^ (tok & 7)) << 4), w[ti][0], w[ti][1], w[ti][2], w[ti][3]);
                        if (tok >= nvalid) w[ti][0] = w[ti][1] = w[ti][2] = w[ti][3] = 0u;
                    }
#pragma unroll
                    for (int jj = 0; jj < 8; ++jj) {
                        const uint32_t sel = (jj & 1) ? 0x7362u : 0x5140u;
                        const uint32_t x01 = prmt(w[0][jj >> 1], w[1][jj >> 1], sel), x23 = prmt(w[2][jj >> 1], w[3][jj >> 1], sel);
                        const uint32_t a0 = e4m3x2_to_f16x2(x01 & 0xffff), a1 = e4m3x2_to_f16x2(x01 >> 16);
                        const uint32_t a2 = e4m3x2_to_f16x2(x23 & 0xffff), a3 = e4m3x2_to_f16x2(x23 >> 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][jj], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(b_free + 8 * st);
        }
        // ---------------- the warps' states, joined: 3 into 2, into 1, into 0
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[nt][e];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                l[nt][e] = v;
            }
        // a state in shared memory: a float4 a lane for each (n-tile, j), then (max, sum) of
        // the lane's columns
        auto put = [&]() {
            float4 *to = reinterpret_cast<float4 *>(smem + LY::S_JOIN);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int jj = 0; jj < 8; ++jj)
                    to[(nt * 8 + jj) * 32 + lane] = make_float4(o[nt][jj][0], o[nt][jj][1], o[nt][jj][2], o[nt][jj][3]);
            float *ml = reinterpret_cast<float *>(to + NT * 8 * 32);
            if (gq == 0)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        ml[2 * (nt * 8 + 2 * cq + e)] = m[nt][e];
                        ml[2 * (nt * 8 + 2 * cq + e) + 1] = l[nt][e];
                    }
        };
        auto add = [&]() {
            const float4 *from = reinterpret_cast<const float4 *>(smem + LY::S_JOIN);
            const float *ml = reinterpret_cast<const float *>(from + NT * 8 * 32);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float f0[2], f1[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float m1 = ml[2 * (nt * 8 + 2 * cq + e)], l1 = ml[2 * (nt * 8 + 2 * cq + e) + 1];
                    const float M = fmaxf(m[nt][e], m1), R = M == -INFINITY ? 0.f : M;
                    f0[e] = ex2(m[nt][e] - R);
                    f1[e] = ex2(m1 - R);
                    m[nt][e] = M;
                    // (sums that are not numbers stay so, with no score to be the largest too)
                    l[nt][e] = M == -INFINITY ? l[nt][e] + l1 : f0[e] * l[nt][e] + f1[e] * l1;
                }
#pragma unroll
                for (int jj = 0; jj < 8; ++jj) {
                    const float4 v = from[(nt * 8 + jj) * 32 + lane];
                    o[nt][jj][0] = f0[0] * o[nt][jj][0] + f1[0] * v.x;
                    o[nt][jj][1] = f0[1] * o[nt][jj][1] + f1[1] * v.y;
                    o[nt][jj][2] = f0[0] * o[nt][jj][2] + f1[0] * v.z;
                    o[nt][jj][3] = f0[1] * o[nt][jj][3] + f1[1] * v.w;
                }
            }
        };
        // (the last warp's turn comes when warp 0 has read the item before)
        if (warp < CONSUMERS - 1) {
            if (!wait(b_join + 8 * (warp + 1), k)) return;
            add();
        } else if (k > 0 && !wait(b_join, k - 1)) {
            return;
        }
        __syncwarp();
        if (warp > 0) put();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_join + 8 * warp);
        if (warp > 0) continue;
        // ---------------- warp 0 has the item's result
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = nt * 8 + 2 * cq + e;
                if (c >= cols) continue;
                const size_t rh = (size_t)(it.row0 + c / p.group) * p.hq + it.g * p.group + c % p.group;
                if (p.out16) {
                    const float inv = vsc / l[nt][e];     // (a sum of 0: scores that are all -inf, NaN)
                    __nv_bfloat16 *to = p.out16 + rh * D;
#pragma unroll
                    for (int jj = 0; jj < 8; ++jj)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            to[FP8 ? 16 * gq + 2 * jj + i : 16 * jj + gq + 8 * i] = __float2bfloat16(o[nt][jj][e + 2 * i] * inv);
                } else {
                    const size_t pi = rh * p.part_stride + it.slot;
                    float *to = p.part_o + pi * D;
#pragma unroll
                    for (int jj = 0; jj < 8; ++jj)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            to[FP8 ? 16 * gq + 2 * jj + i : 16 * jj + gq + 8 * i] = o[nt][jj][e + 2 * i] * vsc;
                    if (gq == 0)
                        *reinterpret_cast<float2 *>(p.part_ml + pi * 2) = make_float2(l[nt][e] > 0.f ? m[nt][e] : -INFINITY, l[nt][e]);
                }
            }
    }
}

__global__ void set_counter_kernel(int *counter, int to)
{
    griddep_launch_dependents();
    griddep_wait();
    if (threadIdx.x == 0) *counter = to;
}

template <bool FP8, int NT>
cudaError_t launch(const CUtensorMap &km, const CUtensorMap &vm, TailParams p, int *counter, int64_t items, cudaStream_t st)
{
    using LY = TailLay<FP8, NT>;
    const cudaError_t e = pkv_host::ensure_dynamic_smem<shared_tail_kernel<FP8, NT>>(LY::SMEM);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(items, 152 * LY::CTAS));
    if (p.beside) p.counter = counter;       // (set by the kernel of the prefixes)
    else if (counter && items > grid) {
        const cudaError_t set = pkv_host::launch_ex(set_counter_kernel, dim3(1), dim3(32), 0, st, true, counter, grid);
        if (set != cudaSuccess) return set;
        p.counter = counter;
    }
    return pkv_host::launch_ex(shared_tail_kernel<FP8, NT>, dim3(grid), dim3(LY::THREADS), LY::SMEM, st, true, km, vm, p);
}

}  // namespace

namespace pkv_shared_tail {
cudaError_t status_word(uint32_t **at) { return cudaGetSymbolAddress(reinterpret_cast<void **>(at), g_status); }

cudaError_t launch_tails(const SharedCall &c, bool beside, cudaStream_t st)
{
    TailParams p{};
    p.b = c.b;
    p.out16 = shared_parts(c) == 1 ? static_cast<__nv_bfloat16 *>(c.out) : nullptr;
    p.q = c.q;
    p.block_tables = c.block_tables;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.part_o = c.part_o;
    p.part_ml = c.part_ml;
    p.direct = c.tail_splits == 1 && c.sets == 1 ? 1 : 0;
    p.first = beside ? 0 : 1;
    p.hq = c.hq;
    p.hkv = c.hkv;
    p.group = c.hq / c.hkv;
    p.num_blocks = c.num_blocks;
    p.part_blocks = c.tail_part_blocks;
    p.fine_from = c.fine_from;
    p.fine_blocks = c.fine_blocks;
    p.part_stride = shared_parts(c);
    p.part_off = c.prefix_splits;
    p.whole = c.whole ? 1 : 0;
    for (p.set_log2 = 0; 1 << p.set_log2 < c.set_rows;) ++p.set_log2;
    p.beside = beside ? 1 : 0;
    p.scale_log2 = c.scale_log2;
    // bf16: a tile's two 64-dim halves as one box: dims (64 dims, rows, halves), strides
    // (row 256 B, half 128 B); fp8: a tile is one box of 128-byte rows
    const uint64_t rows = (uint64_t)c.num_blocks * c.hkv * BS;
    CUtensorMap map[2];
    for (int i = 0; i < 2; ++i) {
        const void *cache = i ? c.v_cache : c.k_cache;
        if (!(c.fp8 ? pkv_host::encode_tmap_2d(&map[i], cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, D, rows, D, D, BS,
                                               CU_TENSOR_MAP_SWIZZLE_128B)
                    : pkv_host::encode_tmap_3d(&map[i], cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 64, rows, 2, D * 2, 128, 64,
                                               BS, 2, CU_TENSOR_MAP_SWIZZLE_128B)))
            return cudaErrorInvalidValue;
    }
    const int64_t items = tail_kernel_items(c);
    p.most = (int)items;
    int *const counter = p.out16 ? nullptr : c.counter;     // (no workspace where the only part is the output)
    if (std::min(c.b.max_q_len, c.set_rows) * p.group > 8)
        return c.fp8 ? launch<true, 2>(map[0], map[1], p, counter, items, st)
                     : launch<false, 2>(map[0], map[1], p, counter, items, st);
    return c.fp8 ? launch<true, 1>(map[0], map[1], p, counter, items, st)
                 : launch<false, 1>(map[0], map[1], p, counter, items, st);
}

}  // namespace pkv_shared_tail
