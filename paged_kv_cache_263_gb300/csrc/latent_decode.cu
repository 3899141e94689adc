// latent_decode.cu -- attention over a paged latent cache, absorbed form
// (sm_103a, 5th-generation tensor cores, thread-block clusters).
//
// A cached row x_t holds a token's latent (512) and rotary key (64); a head's
// query, multiplied by that head's key expansion beforehand, is 576 wide, and
//   out[r][h] = sum_t p_t x_t[0:512],  p = softmax_t(scale * q[r][h] . x_t)
// over the keys t <= L - n + i that row i of a sequence's n rows sees.
//
// What bounds it.  A key is 1,152 bytes, read once for all heads; a (row, head)
// costs 2 x (576 + 512) operations a key.  One token of 128 heads makes 242
// operations a byte, just under the GPU's ratio (1,916 TFLOP/s : 6,789 GB/s =
// 282), so decode is bound by memory as long as the products run on the tensor
// cores with full tiles: a sequence's (row, head) pairs in units of 128, padded with
// zero rows when there are fewer.  (A unit may begin and end within a row: 12 chunks
// of 70 rows x 96 heads take 117 us; in units of whole rows they took 140.)
//
// Why a pair of CTAs.  The output of 128 rows is 128 x 512 fp32, all of one SM's
// tensor memory, and the queries (144 KiB) and a key tile do not fit its shared
// memory together.  A cluster of two CTAs therefore shares a tile by dims:
// CTA c holds latent dims 256c .. 256c+255 and rotary dims 32c .. 32c+31 of the
// queries and of every key, so that each byte is loaded by one CTA only.
//  * S = Q K^T: each CTA multiplies its 288 dims, giving a partial S[128 x 64]
//    of the 64-key tile; the partial sums (fp32) are exchanged through
//    distributed shared memory (asynchronous stores that count on the receiver's
//    mbarrier) and both CTAs add the two -- a + b is the same either way round,
//    so both hold the same scores.
//  * Each computes the softmax of all 128 rows, and O[128 x 256] += P V over its
//    own 256 dims: the key tile in shared memory is the K-major B operand of the
//    first product and the MN-major B operand of the second.
//  * Tensor memory, 512 columns: Q 96 (192 dims as the A operand of the first
//    product; the other 64 and the rotary part are in shared memory), P 32 (bf16,
//    the A operand of the second product), S 2 x 64, O 256.  P has its own
//    columns so that an S buffer is free as soon as it has been read: the first
//    products run ahead of the softmax.  With P written over S (and all of Q in
//    tensor memory) a tile took 2,000-2,800 cycles, all of it the latency of the
//    loop S -> exchange -> softmax -> PV -> next S over two buffers.
//  * The exchange goes in slots of 32 columns (two of 16 KiB), each released
//    as soon as it is added: a tile is in the slots while the next is multiplied.
//  * Warps 0-7: exchange, softmax and epilogue, one query row a thread; warps 0-3
//    take the even tiles (S buffer 0), warps 4-7 the odd ones, and hand the
//    running maximum on through shared memory.  A tile costs its warps about
//    4,000 cycles, nearly all latency, so one group alone would set the pace.  The
//    group that does not have an item's last tile loads the next item's queries.
//    Warp 8: TMA producer, four stages of 64 keys (36 KiB).  Warps 9 and 10: MMA
//    issuers.
//  * A stage is held for 10,500 cycles -- 4,000 until it has landed, 1,100 for S,
//    4,000 for exchange and softmax, 1,100 for PV -- so four of them give a tile
//    every 2,650, where its bytes need 1,570 and its products 1,090.  (64
//    sequences of 1,500 to 8,200 tokens x 128 heads: 118 us, 3.2 TB/s.  Three stages
//    made it 16 % slower; a ring of four and a half in halves of 32 keys 5 %, for its
//    second set of waits and products; blocks brought into L2 two tiles ahead 2 %.)
//  * The sum that a row is divided by adds its probabilities as fp32, before their
//    rounding to bf16 for the second product.  Both errors are roundings of a
//    probability; adding the rounded ones instead would cancel part of them and costs
//    1 % here.  (Relative RMS error of the output, emulated: 1,000 keys, scores spread
//    by 1.7: 2.28e-3 and 2.21e-3, of which the output's own rounding is 1.64e-3; spread
//    by 5: 2.30e-3 and 1.84e-3.)
//
// Work split.  The tiles of all (sequence, 128-row unit) pairs are laid end to
// end and cut into equal ranges, one a cluster: the batch's ragged lengths
// balance without a plan on the host, and one long context is split over all
// SMs.  A unit that a cut falls into leaves fp32 partial sums in the workspace
// (at most two a cluster), which latent_merge_kernel joins in cluster order.
#include "latent_work.cuh"
#include "trace.h"

#include <algorithm>
#include <cmath>

namespace pkv_latent_small {
kv_status launch(const void *params, const void *q, const void *cache, cudaStream_t st);
}

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float RESCALE_LOG2 = 8.0f;
constexpr int HALF = LAT / 2, RHALF = ROPE / 2;   // a CTA's latent and rotary dims
constexpr int NCL = pkv_split::PAIR.workers;      // clusters: a pair of CTAs on each pair of the 152 SMs
constexpr int STAGES = 4;
constexpr uint32_t CHUNK_BYTES = TK * 128;        // 64 keys x 64 dims
constexpr uint32_t ROPE_OFF = 4 * CHUNK_BYTES;    // within a stage
constexpr uint32_t STAGE_BYTES = ROPE_OFF + TK * 64;
constexpr int QT = 192;                           // a CTA's query dims in tensor memory; the other 64 are in shared
constexpr uint32_t SQ = STAGES * STAGE_BYTES;     // query dims 192..255 of the CTA's 256, 128 rows x 128 bytes
constexpr uint32_t SQR = SQ + 128 * 128;          // the queries' rotary part, 128 rows x 64 bytes
constexpr int SLOTS = 2, SCOLS = 32;              // the peer's partial scores: slots of 32 columns,
constexpr uint32_t SRECV = SQR + 128 * 64;        // [8 groups of 4 columns][128 rows] float4
constexpr uint32_t SLOT_BYTES = 128 * SCOLS * 4;
constexpr uint32_t SMAX = SRECV + SLOTS * SLOT_BYTES;   // running maxima [128]; at an item's end [item parity][group](sum, maximum)[128]
constexpr uint32_t SBAR = SMAX + 9 * 128 * 4;
constexpr uint32_t LIST_OFF = 512;                // within the barrier area
constexpr int LIST = 40;                          // sequences tabled in shared memory
constexpr int SMEM_BYTES = SBAR + 1024 + 1024;    // + 1 KiB: aligned to 1 KiB at run time
constexpr int W_PROD = 8, W_MMA = 9, THREADS = 32 * (W_MMA + 2);
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");

enum {
    B_KVF = 0,                  // + stage: the tile landed
    B_KVE = B_KVF + STAGES,     // + stage: every MMA reading it is done
    B_Q = B_KVE + STAGES,       // the item's queries are in place (128 arrivals)
    B_S = B_Q + 1,              // + buffer: a partial S tile is in tensor memory
    B_SFREE = B_S + 2,          // + buffer: it has been read (a group's 4 warps)
    B_RECV = B_SFREE + 2,       // + 4 x slot + row warp: the peer's partial rows arrived
    B_RFREE = B_RECV + 4 * SLOTS,   // + 4 x slot + row warp: the peer has read what this CTA sent
    B_SORD = B_RFREE + 4 * SLOTS,   // + row warp: the tile's partial rows have been sent
    B_MAX = B_SORD + 4,         // + row warp: the peer's have been added, the running maxima are in shared memory
    B_SUM = B_MAX + 4,          // + row warp: both groups' sums are in shared memory
    B_P = B_SUM + 4,            // P is in tensor memory (128 arrivals)
    B_PVD = B_P + 1,            // + tile parity: its PV product finished (one barrier each: a group waits for
                                // every second tile's, and a parity must not be waited for two phases ahead)
    B_DRAIN = B_PVD + 2,        // every MMA of the item finished
    B_OFREE = B_DRAIN + 1,      // the item's O was read (256 arrivals)
    B_END = B_OFREE + 1,        // + issuer: everything it issued finished
    NBAR = B_END + 2
};
static_assert(QT == 192, "the loads of the queries");
static_assert(NBAR * 8 + 64 <= LIST_OFF && LIST_OFF + LIST * 12 <= 1024, "barrier area");

// instruction descriptors, kind::f16: bf16 A and B, fp32 accumulate, M = 128
constexpr uint32_t idesc(int n, bool b_mn_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn_major ? (1u << 16) : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}
constexpr uint32_t IDESC_S = idesc(TK, false);
constexpr uint32_t IDESC_PV = idesc(HALF, true);

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes into the peer's shared memory, counted on the peer's mbarrier
__device__ __forceinline__ void st_async_v4(uint32_t addr, float a, float b, float c, float d, uint32_t bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(addr),
                 "f"(a), "f"(b), "f"(c), "f"(d), "r"(bar)
                 : "memory");
}
// tells the peer that this warp has read what it sent: after a __syncwarp, which
// orders the other lanes' reads before it.  The release is at CTA scope on purpose.
// What has to be done before are this warp's reads of this SM's own shared memory,
// and a read of it that is done for the CTA is done for everybody; a release at
// cluster scope waits for the SM's other memory traffic as well (64 sequences of
// 1,500 to 8,200 tokens x 128 heads: 118 us with this one, 176 with that, 165 with
// that one in a warp of its own).
__device__ __forceinline__ void arrive_peer(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 64-byte-swizzled K-major operand (rows of 64 bytes)
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t sbo_bytes)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)((sbo_bytes >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)4 << 61;
    return d;
}

__global__ void __launch_bounds__(THREADS, 1) __cluster_dims__(2, 1, 1)
    latent_kernel(const __grid_constant__ CUtensorMap lmap, const __grid_constant__ CUtensorMap rmap,
                  const LatentParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SBAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NBAR);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *s_start = reinterpret_cast<int *>(tmem_slot + 2);        // the range's first sequence, unit and tile
    int *s_work = reinterpret_cast<int *>(bars + NBAR + 4);   // the cut: each, extra
    int *list = reinterpret_cast<int *>(smem + SBAR + LIST_OFF);
    int *scan = reinterpret_cast<int *>(smem + SMAX);         // setup only
    auto bar = [&](int i) -> uint32_t { return sbase + SBAR + i * 8; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t c = cluster_rank(), peer = c ^ 1u;
    const int k = blockIdx.x >> 1;                                // cluster
    griddep_launch_dependents();

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(bar(B_KVF + i), 1);
            mbar_init(bar(B_KVE + i), 1);
        }
        mbar_init(bar(B_Q), 128);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_SFREE + i), 4);
            mbar_init(bar(B_END + i), 1);
        }
        for (int i = 0; i < 4 * SLOTS; ++i) {
            mbar_init(bar(B_RECV + i), 1);
            mbar_init(bar(B_RFREE + i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(B_SORD + i), 1);
            mbar_init(bar(B_MAX + i), 1);
            mbar_init(bar(B_SUM + i), 2);
        }
        mbar_init(bar(B_P), 128);
        mbar_init(bar(B_PVD), 1);
        mbar_init(bar(B_PVD + 1), 1);
        mbar_init(bar(B_DRAIN), 1);
        mbar_init(bar(B_OFREE), 256);
        *abort_flag = 0;
        s_start[0] = p.num_seqs;
        s_start[1] = s_start[2] = 0;
        fence_mbar_init();
        prefetch_tmap(&lmap);
        prefetch_tmap(&rmap);
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();      // the barriers exist: the peer may use them once it has waited for this CTA
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    griddep_wait();       // everything below reads what earlier kernels wrote
    constexpr pkv_split::Rule rule = pkv_split::PAIR;
    const Range range = find_range<THREADS>(p, rule, k, blockIdx.x == 0, scan, s_start, s_work, list, LIST);
    Walk walk = range.walk;
    tc_fence_after();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // the peer's barriers exist
    const uint32_t tmem = *tmem_slot;
    const uint32_t tQ = tmem, tP = tmem + QT / 2, tO = tmem + 256;
    auto tS = [&](int b) -> uint32_t { return tmem + 128 + b * TK; };

    Item it;
    if (warp == W_PROD) {
        // ======================= producer: a box of a block's 16 keys x 64 (or 32 rotary)
        // dims at a time, issued by one elected lane; each lane reads the id of block
        // lane % 4 of the next tile while it waits for the stage
        const int blk = lane & 3;
        int u = 0;
        bool ok = true;
        while (ok && next_item(p, range, walk, it)) {
            const int32_t *bt = p.tables + (size_t)it.s * p.max_blocks;
            const int nblk = (it.q.L + BS - 1) / BS;
            // the item's queries, into L2 (this warp runs up to four tiles ahead; the
            // first item's are being loaded already)
            for (int r = lane; u > 0 && r < it.rows; r += 32) {
                const uint16_t *src = p.q + ((size_t)it.q.a * p.heads + it.r0 + r) * LKD;
#pragma unroll
                for (int e = 0; e < 4; ++e) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + c * HALF + e * 64));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(src + LAT + c * RHALF));
            }
            __syncwarp();
            auto block_id = [&](int j) -> int32_t {
                const int b = j * (TK / BS) + blk;
                return (j < it.j1 && b < nblk) ? __ldg(bt + b) : -1;
            };
            int32_t next_id = block_id(it.j0);
            for (int j = it.j0; j < it.j1; ++j, ++u) {
                const int st = u % STAGES;
                const int32_t id = next_id;
                next_id = block_id(j + 1);
                if (u >= STAGES && !wait_bar(bar(B_KVE + st), ((u - STAGES) / STAGES) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const bool in = j * (TK / BS) + blk < nblk;
                const bool valid = in && id >= 0 && id < p.num_blocks;
                if (in && !valid && lane < 4) flag(ST_BAD_BLOCK);
                const unsigned vm = __ballot_sync(0xffffffffu, valid) & 15u;
                int32_t rows[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) rows[b] = __shfl_sync(0xffffffffu, id, b) * BS;
                if (elect_one()) {
                    fence_proxy_async_smem();
                    mbar_arrive_expect_tx(bar(B_KVF + st), __popc(vm) * (4 * 2048 + 1024));
                    const uint32_t stg = sbase + st * STAGE_BYTES;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (!(vm >> b & 1)) continue;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            tma_load_2d(stg + e * CHUNK_BYTES + b * 2048, &lmap, c * HALF + e * 64, rows[b], bar(B_KVF + st));
                        tma_load_2d(stg + ROPE_OFF + b * 1024, &rmap, LAT + c * RHALF, rows[b], bar(B_KVF + st));
                    }
                }
                __syncwarp();
            }
        }
        if (*abort_flag)      // loads in flight land before the CTA exits
            for (int uu = max(0, u - STAGES); uu < u; ++uu)
                (void)mbar_wait_bounded(bar(B_KVF + uu % STAGES), (uu / STAGES) & 1);
    } else if (warp >= W_MMA) {
        // ======================= MMA issuers: one warp the first product of every
        // tile, the other the second, so that a second product never queues behind
        // a first one whose tile has not landed.  One elected lane issues: with
        // elect.sync the compiler keeps descriptors in uniform registers, and a
        // 128 x 64 x 16 product leaves every 33 cycles (54 from a lane-0 branch,
        // measured), which is its execution time.
        int x = 0, items = 0;       // tiles and items done
        bool ok = true;
        if (warp == W_MMA) {
            const uint64_t kdesc0 = sdesc_sw128(sbase, 16, 1024);
            const uint64_t rdesc0 = sdesc_sw64(sbase + ROPE_OFF, 512);
            const uint64_t qdesc = sdesc_sw128(sbase + SQ, 16, 1024), qrdesc = sdesc_sw64(sbase + SQR, 512);
            for (; ok && next_item(p, range, walk, it); ++items) {
                ok = wait_bar(bar(B_Q), items & 1, abort_flag);
                for (int j = it.j0; ok && j < it.j1; ++j, ++x) {
                    const int st = x % STAGES, b = x & 1;
                    // S(x - 2) has been read
                    if (x >= 2 && !wait_bar(bar(B_SFREE + b), ((x >> 1) - 1) & 1, abort_flag)) { ok = false; break; }
                    if (!wait_bar(bar(B_KVF + st), (x / STAGES) & 1, abort_flag)) { ok = false; break; }
                    const int first = it.q.L - j * TK;
                    if (first < TK) {
                        // keys at or past the context's end may hold anything (never
                        // written, or not loaded); P is 0 there, but 0 x NaN is NaN
                        const uint32_t vb = sbase + st * STAGE_BYTES;
                        for (int e = lane; e < (TK - first) * 32; e += 32)
                            st_shared_v4(vb + ((e >> 3) & 3) * CHUNK_BYTES + (first + (e >> 5)) * 128 + (e & 7) * 16, 0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (elect_one()) {
                        tc_fence_after();
                        const uint64_t off = (uint64_t)((st * STAGE_BYTES) >> 4);
                        const uint32_t ts = tS(b);
#pragma unroll
                        for (int kk = 0; kk < QT / 16; ++kk)
                            umma_f16_ts(ts, tQ + kk * 8, kdesc0 + off + (uint64_t)(((kk >> 2) * CHUNK_BYTES + (kk & 3) * 32) >> 4),
                                        IDESC_S, kk > 0);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16(ts, qdesc + (uint64_t)((kk * 32) >> 4),
                                     kdesc0 + off + (uint64_t)((3 * CHUNK_BYTES + kk * 32) >> 4), IDESC_S, 1u);
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk)
                            umma_f16(ts, qrdesc + (uint64_t)((kk * 32) >> 4), rdesc0 + off + (uint64_t)((kk * 32) >> 4), IDESC_S, 1u);
                        umma_commit(bar(B_S + b));
                    }
                    __syncwarp();
                }
            }
        } else {
            const uint64_t vdesc0 = sdesc_sw128(sbase, CHUNK_BYTES, 1024);
            for (; ok && next_item(p, range, walk, it); ++items) {
                for (int j = it.j0; j < it.j1; ++j, ++x) {
                    const int st = x % STAGES;
                    // the item before: its O has been read
                    if (j == it.j0 && items > 0 && !wait_bar(bar(B_OFREE), (items - 1) & 1, abort_flag)) { ok = false; break; }
                    if (!wait_bar(bar(B_P), x & 1, abort_flag)) { ok = false; break; }
                    if (elect_one()) {
                        tc_fence_after();
                        const uint64_t vd = vdesc0 + (uint64_t)((st * STAGE_BYTES) >> 4);
#pragma unroll
                        for (int kk = 0; kk < TK / 16; ++kk)
                            umma_f16_ts(tO, tP + kk * 8, vd + (uint64_t)((kk * 2048) >> 4), IDESC_PV, (j > it.j0 || kk > 0) ? 1u : 0u);
                        umma_commit(bar(B_PVD + (x & 1)));
                        umma_commit(bar(B_KVE + st));
                        if (j == it.j1 - 1) umma_commit(bar(B_DRAIN));
                    }
                    __syncwarp();
                }
            }
        }
        // everything issued has finished before tensor memory is released
        if (elect_one()) umma_commit(bar(B_END + (warp - W_MMA)));
        __syncwarp();
        (void)mbar_wait_bounded(bar(B_END + (warp - W_MMA)), 0);
    } else {
        // ======================= exchange, softmax and epilogue: threads r (even
        // tiles) and r + 128 (odd tiles) = query row r
        const int r = threadIdx.x & 127, w = warp & 3, grp = warp >> 2;
        const uint32_t lane_base = (uint32_t)(w * 32) << 16;
        volatile float *m_sh = reinterpret_cast<volatile float *>(smem + SMAX), *l_sh = m_sh + 128;
        int x = 0, items = 0, hs = 0;         // tiles, items, slots of the exchange so far
        int sums = 0;                         // items this warp had a real row in
        const float sl = p.scale_log2;
        bool merges = false;
        // an item's queries, into tensor and shared memory.  A row is a lane of
        // tensor memory, but 16 bytes of 32 rows in one load would touch 32 lines
        // (that took 6,400 cycles): 8 lanes read 128 bytes of a row, and the warp's
        // part of the shared query tile turns them round, 64 dims at a time
        auto load_queries = [&]() {                       // of the item that follows
            Walk ahead = walk;
            Item q;
            if (!next_item(p, range, ahead, q)) return;
            const int rows = q.rows;
            const uint16_t *src = p.q + ((size_t)q.q.a * p.heads + q.r0 + w * 32) * LKD;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            const int lr = lane >> 3, le = lane & 7;      // row within four, piece
            const uint32_t qt = sbase + SQ + w * 4096;
            uint4 y[2][8];
            auto fetch = [&](int h, uint4 (&v)[8]) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = w * 32 + 4 * i + lr < rows
                               ? __ldg(reinterpret_cast<const uint4 *>(src + (size_t)(4 * i + lr) * LKD + c * HALF + h * 64) + le) : zero;
            };
            fetch(0, y[0]);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                if (h < 3) {
                    fetch(h + 1, y[(h + 1) & 1]);
                } else {
                    // the rotary part: 4 lanes read a row's 64 bytes
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[0][i] = w * 32 + 8 * i + (lane >> 2) < rows
                                      ? __ldg(reinterpret_cast<const uint4 *>(src + (size_t)(8 * i + (lane >> 2)) * LKD + LAT + c * RHALF) + (lane & 3)) : zero;
                }
                // (128-byte swizzle: 16-byte pieces permuted by the row's bits 0-2)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = 4 * i + lr;
                    const uint4 t = y[h & 1][i];
                    st_shared_v4(qt + row * 128 + ((le ^ (row & 7)) << 4), t.x, t.y, t.z, t.w);
                }
                __syncwarp();
                if (h < 3) {
                    uint32_t v[32];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        lds128(qt + lane * 128 + ((e ^ (lane & 7)) << 4), v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    tmem_st32u(tQ + lane_base + 32 * h, v);
                    __syncwarp();
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = w * 32 + 8 * i + (lane >> 2);
                // (64-byte swizzle: by the row's bits 1-2)
                st_shared_v4(sbase + SQR + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4), y[0][i].x, y[0][i].y, y[0][i].z, y[0][i].w);
            }
            tmem_wait_st();
            tc_fence_before();
            fence_proxy_async_smem();
            mbar_arrive(bar(B_Q));
        };
        bool ok = true;
        if (grp == 1) load_queries();
        while (ok && next_item(p, range, walk, it)) {
            const int rows = it.rows;
            const bool active = w * 32 < rows;
            const int first_pos = it.q.L - it.q.n + (int)((uint32_t)it.r0 / (uint32_t)p.heads);
            const int tok = (int)((uint32_t)(it.r0 + min(r, rows - 1)) / (uint32_t)p.heads - (uint32_t)it.r0 / (uint32_t)p.heads);
            const int pos = it.q.L > 0 ? first_pos + tok : -1;    // the last key this row sees
            const int pos_min = it.q.L > 0 ? first_pos : -1;
            float m_ref = -INFINITY, l = 0.f;                     // (l relative to m_ref)
            for (int j = it.j0; j < it.j1; ++j, ++x, hs += active ? TK / SCOLS : 0) {
                if ((x & 1) != grp) continue;
                const int t0 = j * TK;
                if (!wait_bar(bar(B_S + grp), (x >> 1) & 1, abort_flag)) { ok = false; break; }
                float sv[TK];
                if (active) {
                    tc_fence_after();
                    tmem_ld64(tS(grp) + lane_base, sv);
                    tc_fence_before();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(bar(B_SFREE + grp));
                // (the groups send, and add, their tiles in turn: a slot's phases would
                // otherwise be waited for out of order, which a parity cannot tell)
                if (x > 0 && !wait_bar(bar(B_SORD + w), (x - 1) & 1, abort_flag)) { ok = false; break; }
                float mraw = -INFINITY;
                if (active) {
                    // this CTA's part of the sums to the peer, 32 columns at a time
#pragma unroll
                    for (int h = 0; h < TK / SCOLS; ++h) {
                        const int slot = (hs + h) % SLOTS, i = 4 * slot + w;
                        if (hs + h >= SLOTS && !wait_bar<true>(bar(B_RFREE + i), ((hs + h) / SLOTS - 1) & 1, abort_flag)) ok = false;
                        const uint32_t dst = peer_addr(sbase + SRECV + slot * SLOT_BYTES + r * 16, peer);
                        const uint32_t rb = peer_addr(bar(B_RECV + i), peer);
                        if (ok) {
#pragma unroll
                            for (int e = 0; e < SCOLS; e += 4)
                                st_async_v4(dst + e * 512, sv[h * SCOLS + e], sv[h * SCOLS + e + 1], sv[h * SCOLS + e + 2],
                                            sv[h * SCOLS + e + 3], rb);
                        }
                    }
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(bar(B_SORD + w));
                // the running maximum after the tile before
                if (x > 0 && !wait_bar(bar(B_MAX + w), (x - 1) & 1, abort_flag)) ok = false;
                if (!ok) break;
                if (active) {
                    // the peer's part
#pragma unroll
                    for (int h = 0; h < TK / SCOLS; ++h) {
                        const int slot = (hs + h) % SLOTS, i = 4 * slot + w;
                        if (lane == 0) mbar_arrive_expect_tx(bar(B_RECV + i), 32 * SCOLS * 4);
                        if (!wait_bar<true>(bar(B_RECV + i), ((hs + h) / SLOTS) & 1, abort_flag)) ok = false;
                        const uint32_t src = sbase + SRECV + slot * SLOT_BYTES + r * 16;
                        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < SCOLS / 4; ++e) {
                            uint32_t a[4];
                            lds128(src + e * 2048, a[0], a[1], a[2], a[3]);
#pragma unroll
                            for (int f = 0; f < 4; ++f) sv[h * SCOLS + 4 * e + f] += __uint_as_float(a[f]);
                        }
                        if (t0 + h * SCOLS + SCOLS - 1 > pos_min) {
#pragma unroll
                            for (int e = 0; e < SCOLS; ++e)
                                if (t0 + h * SCOLS + e > pos) sv[h * SCOLS + e] = -INFINITY;
                        }
                        // raw scores; the scale (> 0) is applied inside the exponent's FFMA
#pragma unroll
                        for (int e = 0; e < SCOLS; e += 8)
#pragma unroll
                            for (int f = 0; f < 4; ++f) m4[f] = max3(m4[f], sv[h * SCOLS + e + f], sv[h * SCOLS + e + 4 + f]);
                        mraw = max3(mraw, fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    }
                    if (!ok) break;
                }
                float alpha = 1.f, beta = 1.f;
                if (active) {
                    const float m_old = j > it.j0 ? m_sh[r] : -INFINITY;
                    const float mx = mraw * sl;
                    // the reference moves only when the maximum has grown by 2^8 (P stays
                    // finite in fp32 and bf16, whose relative precision does not depend on
                    // its size): O is seldom rescaled
                    float m_new = m_old;
                    if (mx > m_old + RESCALE_LOG2 || (m_old == -INFINITY && mx != -INFINITY)) {
                        alpha = m_old == -INFINITY ? 0.f : ex2(m_old - mx);
                        m_new = mx;
                    }
                    if (m_new != m_ref) beta = m_ref == -INFINITY ? 0.f : ex2(m_ref - m_new);
                    m_ref = m_new;
                    m_sh[r] = m_new;
                    __syncwarp();
                }
                if (lane == 0) {
                    mbar_arrive(bar(B_MAX + w));
#pragma unroll
                    for (int h = 0; h < TK / SCOLS; ++h)
                        if (active) arrive_peer(peer_addr(bar(B_RFREE + 4 * ((hs + h) % SLOTS) + w), peer));
                }
                if (active) {
                    const bool rescale = __any_sync(0xffffffffu, alpha != 1.f);
                    const float mneg = m_ref == -INFINITY ? 0.f : -m_ref;
                    const uint64_t sl2 = f2_pack(sl, sl), mn2 = f2_pack(mneg, mneg);
                    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
                    uint32_t pw[TK / 2];
#pragma unroll
                    for (int e = 0; e < TK / 2; ++e) {
                        float y0, y1;
                        f2_unpack(f2_fma(f2_pack(sv[2 * e], sv[2 * e + 1]), sl2, mn2), y0, y1);
                        const float p0 = ex2(y0), p1 = ex2(y1);
                        acc[e & 3] = f2_add(acc[e & 3], f2_pack(p0, p1));
                        pw[e] = pack_bf16(p0, p1);   // the second product's operand type, beside bf16 values
                    }
                    float s0, s1;
                    f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
                    l = l * beta + (s0 + s1);
                    // PV(x - 1) has read P and accumulated into O
                    if (x > 0 && !wait_bar(bar(B_PVD + (grp ^ 1)), ((x - 1) >> 1) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    if (j > it.j0 && rescale) {
#pragma unroll 1
                        for (int h = 0; h < HALF / 16; ++h) {
                            float o[16];
                            tmem_ld16(tO + lane_base + h * 16, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= alpha;
                            tmem_st16(tO + lane_base + h * 16, o);
                        }
                    }
                    tmem_st32u(tP + lane_base, pw);
                    tmem_wait_st();
                    tc_fence_before();
                } else if (x > 0 && !wait_bar(bar(B_PVD + (grp ^ 1)), ((x - 1) >> 1) & 1, abort_flag)) {
                    // (a warp without a real row arrives once a tile, too)
                    ok = false;
                    break;
                }
                mbar_arrive(bar(B_P));
            }
            if (!ok) break;
            if (((x - 1) & 1) != grp) {
                // the next item's queries, once the last first product of this one (in
                // the other group's buffer) has finished
                if (!wait_bar(bar(B_S + (grp ^ 1)), ((x - 1) >> 1) & 1, abort_flag)) break;
                load_queries();
            }
            // both groups' sums, each relative to the maximum it last used (a group
            // without a tile: 0 and -inf); the item's maximum is the larger
            if (active) {
                volatile float *mine = l_sh + ((sums & 1) * 4 + 2 * grp) * 128 + r;
                const volatile float *other = l_sh + ((sums & 1) * 4 + 2 * (grp ^ 1)) * 128 + r;
                mine[0] = l;
                mine[128] = m_ref;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_SUM + w));
                if (!wait_bar(bar(B_SUM + w), sums & 1, abort_flag)) break;
                ++sums;
                const float lo = other[0], mo = other[128];
                const float m = fmaxf(m_ref, mo);
                // (without a score above -inf a sum is 0, or NaN if the query was not finite)
                l = (m_ref == -INFINITY ? l : l * ex2(m_ref - m)) + (mo == -INFINITY ? lo : lo * ex2(mo - m));
                m_ref = m;
            }
            if (!wait_bar(bar(B_DRAIN), items & 1, abort_flag)) break;
            tc_fence_after();
            const bool whole = it.whole();
            const int slot = pkv_split::own_slot(k, it);
            if (active) {
                const size_t row0 = (size_t)it.q.a * p.heads + it.r0;
                const size_t pr0 = (size_t)slot * p.unit, pr = pr0 + r;
                const int d0 = c * HALF + grp * (HALF / 2);
                const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
                // 4 lanes exchange their rows' pieces so that they store 64 bytes of one
                // row together (a store of 16 bytes to each of 32 rows touches 32 lines)
#pragma unroll 1
                for (int h = 0; h < HALF / 64; ++h) {
                    float o[32];
                    tmem_ld32(tO + lane_base + grp * (HALF / 2) + h * 32, o);
                    const int r4 = w * 32 + (lane & ~3), e4 = lane & 3;       // the quad's first row, this lane's piece
                    if (whole) {
                        uint32_t v[4][4];
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e >> 2][e & 3] = pack_bf16(o[2 * e] * inv, o[2 * e + 1] * inv);
                        quad_transpose(v, lane);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (r4 + i < rows)
                                reinterpret_cast<uint4 *>(p.out + (row0 + r4 + i) * LAT + d0 + h * 32)[e4] =
                                    make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
                    } else {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            uint32_t v[4][4];
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e >> 2][e & 3] = __float_as_uint(o[16 * g + e]);
                            quad_transpose(v, lane);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (r4 + i < rows)
                                    reinterpret_cast<uint4 *>(p.part_o + (pr0 + r4 + i) * LAT + d0 + h * 32 + g * 16)[e4] =
                                        make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
                        }
                    }
                }
                if (!whole && r < rows && c == 0 && grp == 0) {
                    p.part_ml[2 * pr] = l == 0.f ? -INFINITY : m_ref;
                    p.part_ml[2 * pr + 1] = l;
                }
            }
            tc_fence_before();
            mbar_arrive(bar(B_OFREE));
            if (!whole && it.j0 == 0 && threadIdx.x == 0 && c == 0) {
                list_merge(p, range, it, k, rows);
                merges = true;
            }
            ++items;
        }
        // (the workspace starts with anything)
        if (!merges && threadIdx.x == 0 && c == 0) p.desc[k] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
    cluster_sync_all();   // nothing is sent to a CTA that has left
}

// Joins the partial sums of the units that a cut fell into, worker by worker, with
// weights 2^(m_i - max m).  Bound by latency: the first partial rows are requested
// before the maxima are known, one wave of CTAs does it all (four a SM; with 98
// registers a thread and 1,216 CTAs it took four waves, 19 us behind 113 for 64
// sequences x 128 heads, now 10), and a unit of more than 16 partials -- one long
// context: 24 us, then 10 -- gets a whole CTA a (row, 128 dims) instead of a warp; one of
// more than 4 if there are CTAs for all (1,000 keys, 128 heads: 17.8 us -> 17.2).
constexpr int MERGE_CTAS = 4 * 152, MERGE_WARPS = 8, MERGE_FEW = 4, MERGE_MANY = 16, MERGE_PRE = 4;

__device__ __forceinline__ void merge_add(float4 &acc, float f, const float4 &v)
{
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
}

__global__ void __launch_bounds__(32 * MERGE_WARPS, 4) latent_merge_kernel(const LatentParams p)
{
    __shared__ int before[MAX_WORKERS + 1];      // rows of the units before worker k's: narrow ones + (wide ones << 16)
    __shared__ int parts[MAX_WORKERS];           // partials of worker k's unit
    __shared__ float4 sums[MERGE_WARPS][32];
    __shared__ float factor[MAX_WORKERS], red[2][MERGE_WARPS];
    static_assert(MAX_WORKERS * 128 < 32768 && MAX_WORKERS <= 32 * MERGE_WARPS, "packed sums; a thread a partial");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_launch_dependents();
    griddep_wait();
    if (warp == 0) {
        int4 units[(MAX_WORKERS + 31) / 32];
        int rows = 0, run = 0;
#pragma unroll
        for (int i = 0; i < (MAX_WORKERS + 31) / 32; ++i) {
            units[i] = 32 * i + lane < p.workers ? p.desc[32 * i + lane] : make_int4(0, 0, 0, 0);
            if (!units[i].x) units[i].z = 0;
            rows += units[i].z;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, o);
        const int wide = rows * 4 <= MERGE_CTAS ? MERGE_FEW : MERGE_MANY;
#pragma unroll
        for (int i = 0; i < (MAX_WORKERS + 31) / 32; ++i) {
            const int b = 32 * i;
            const int4 d = units[i];
            const int n = d.y > wide ? d.z << 16 : d.z;
            int v = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += t;
            }
            if (b + lane < p.workers) {
                parts[b + lane] = d.y;
                before[b + lane] = run + v - n;
            }
            run += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) before[p.workers] = run;
    }
    __syncthreads();
    // the worker with the g-th row of a kind: the last one with no more rows before its own
    auto worker = [&](int g, int shift) -> int {
        int k = 0, hi = p.workers;
        while (hi - k > 1) {
            const int mid = (k + hi) >> 1;
            if (((before[mid] >> shift) & 0xffff) <= g) k = mid;
            else hi = mid;
        }
        return k;
    };
    // partial i of worker k's unit
    auto slot = [&](int k, int i) -> size_t { return (size_t)pkv_split::partial_slot(k, i) * p.unit; };
    auto store = [&](int64_t row, int q4, const float4 &a, float l) {
        const float inv = l == 0.f ? 0.f : 1.f / l;       // (NaN stays NaN, also with partial sums left out)
        reinterpret_cast<uint2 *>(p.out + row * LAT + q4 * 128)[lane] = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
    };
    // few partials: a warp a quarter of a row
    const int narrow = (before[p.workers] & 0xffff) * 4;
    for (int t = blockIdx.x * MERGE_WARPS + warp; t < narrow; t += MERGE_CTAS * MERGE_WARPS) {
        const int g = t >> 2, q4 = t & 3, k = worker(g, 0), row = g - (before[k] & 0xffff), ns = parts[k];
        auto part = [&](int i) -> float4 {
            return i < ns ? reinterpret_cast<const float4 *>(p.part_o + (slot(k, i) + row) * LAT + q4 * 128)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        float4 v[MERGE_PRE];
#pragma unroll
        for (int j = 0; j < MERGE_PRE; ++j) v[j] = part(j);
        const float2 e = lane < ns ? *reinterpret_cast<const float2 *>(p.part_ml + 2 * (slot(k, lane) + row)) : make_float2(-INFINITY, 0.f);
        const int64_t row0 = p.desc2[k];
        float M = e.x;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        M = __shfl_sync(0xffffffffu, M, 0);
        const float f = M == -INFINITY ? 0.f : ex2(e.x - M);
        float l = f * e.y;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        l = __shfl_sync(0xffffffffu, l, 0);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = 0; j0 < ns; j0 += MERGE_PRE) {
            if (j0 > 0) {
#pragma unroll
                for (int j = 0; j < MERGE_PRE; ++j) v[j] = part(j0 + j);
            }
#pragma unroll
            for (int j = 0; j < MERGE_PRE; ++j) {
                const float fj = __shfl_sync(0xffffffffu, f, j0 + j);
                if (j0 + j < ns && M != -INFINITY) merge_add(acc, fj, v[j]);
            }
        }
        store(row0 + row, q4, acc, l);
    }
    // more: the CTA takes a quarter of a row, its warps every eighth partial
    const int wide = (before[p.workers] >> 16) * 4;
    for (int t = blockIdx.x; t < wide; t += MERGE_CTAS) {
        const int g = t >> 2, q4 = t & 3, k = worker(g, 16), row = g - (before[k] >> 16), ns = parts[k];
        auto part = [&](int i) -> float4 {
            return i < ns ? reinterpret_cast<const float4 *>(p.part_o + (slot(k, i) + row) * LAT + q4 * 128)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        float4 v[2 * MERGE_PRE];
#pragma unroll
        for (int j = 0; j < 2 * MERGE_PRE; ++j) v[j] = part(warp + j * MERGE_WARPS);
        float2 e = make_float2(-INFINITY, 0.f);
        if (threadIdx.x < ns) e = *reinterpret_cast<const float2 *>(p.part_ml + 2 * (slot(k, threadIdx.x) + row));
        float M = e.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (lane == 0) red[0][warp] = M;
        __syncthreads();
        for (int i = 0; i < MERGE_WARPS; ++i) M = fmaxf(M, red[0][i]);
        const float f = M == -INFINITY ? 0.f : ex2(e.x - M);
        if (threadIdx.x < ns) factor[threadIdx.x] = f;
        float l = f * e.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) red[1][warp] = l;
        __syncthreads();
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = 0; warp + j0 * MERGE_WARPS < ns; j0 += 2 * MERGE_PRE) {
            if (j0 > 0) {
#pragma unroll
                for (int j = 0; j < 2 * MERGE_PRE; ++j) v[j] = part(warp + (j0 + j) * MERGE_WARPS);
            }
#pragma unroll
            for (int j = 0; j < 2 * MERGE_PRE; ++j) {
                const int i = warp + (j0 + j) * MERGE_WARPS;
                if (i < ns && M != -INFINITY) merge_add(acc, factor[i], v[j]);
            }
        }
        sums[warp][lane] = acc;
        __syncthreads();
        if (warp == 0) {
            l = 0.f;
            for (int i = 0; i < MERGE_WARPS; ++i) l += red[1][i];
            for (int i = 1; i < MERGE_WARPS; ++i) merge_add(acc, 1.f, sums[i][lane]);
            store(p.desc2[k] + row, q4, acc, l);
        }
        __syncthreads();      // the shared sums may be the next row's
    }
}

// How a call's work is laid out.  Units of up to 64 rows take a CTA each
// (latent_small.cu), if that is all that an average sequence has; else a pair of
// CTAs takes 128 (a longer chunk's keys are then read half as often).  Pair and one
// CTA, us: 64 sequences of 1,500 to 8,200 tokens x 64 rows 100 and 87, x 16 rows 92
// and 72; 256 of up to 4,096 x 8 rows 161 and 116; 48 of 300 to 6,000 x 64 rows 63
// and 56, x 96 rows 68 and 89, x 128 rows 75 and 96.  (A single sequence of 1,000:
// 14.4 and 15.1, which the host cannot tell: the lengths are on the device.)
struct Plan {
    bool small;
    int unit, workers;
    size_t desc2, ml, o, total;    // workspace: merge list, partial sums, partial outputs
};
Plan plan(bool small)
{
    Plan y;
    y.small = small;
    y.workers = (small ? pkv_split::ONE : pkv_split::PAIR).workers;
    y.unit = (small ? pkv_split::ONE : pkv_split::PAIR).unit;
    y.desc2 = y.workers * sizeof(int4);
    y.ml = 4096;
    y.o = y.ml + (((size_t)2 * y.workers * y.unit * 8 + 255) & ~(size_t)255);
    y.total = y.o + (size_t)2 * y.workers * y.unit * LAT * 4;
    return y;
}
static_assert(MAX_WORKERS * (sizeof(int4) + 8) <= 4096, "merge list");
static_assert(MAX_WORKERS == 2 * NCL, "both layouts take the same workspace");

}  // namespace

namespace pkv_latent {
cudaError_t status_word(uint32_t **at) { return cudaGetSymbolAddress(reinterpret_cast<void **>(at), g_status); }
}  // namespace pkv_latent

extern "C" {

size_t paged_latent_attention_workspace_size(int32_t num_seqs, int32_t total_q_tokens, int32_t num_heads,
                                             int32_t max_blocks_per_seq)
{
    if (num_seqs < 1 || total_q_tokens < 1 || num_heads < 1 || num_heads > PAGEDKV_LATENT_MAX_HEADS ||
        max_blocks_per_seq < 1)
        return 0;
    return plan(false).total;
}

kv_status paged_latent_attention(void *out, const void *q, const int32_t *cu_q_lens, const int32_t *context_lens,
                                 int32_t num_seqs, int32_t total_q_tokens, const void *cache,
                                 const int32_t *block_tables, int32_t max_blocks_per_seq, int32_t num_heads,
                                 int32_t num_blocks, float scale, void *workspace, size_t workspace_bytes,
                                 void *stream)
{
    PKV_NVTX_RANGE("paged_latent_attention");
    if (num_seqs < 0 || total_q_tokens < 0) return KV_ERR_INVALID;
    if (num_seqs == 0 || total_q_tokens == 0) return KV_OK;
    if (num_heads < 1 || max_blocks_per_seq < 1 || num_blocks < 1) return KV_ERR_INVALID;
    // (key positions are counted in 32 bits, up to the end of a context's last tile)
    if (num_heads > PAGEDKV_LATENT_MAX_HEADS || max_blocks_per_seq > (INT32_MAX - TK + 1) / BS || num_blocks > INT32_MAX / BS)
        return KV_ERR_UNSUPPORTED;
    if (!out || !q || !context_lens || !cache || !block_tables) return KV_ERR_INVALID;
    // (tiles are counted in 32 bits)
    if (((double)total_q_tokens + num_seqs) * (max_blocks_per_seq / (TK / BS) + 1) > 2147483647.0) return KV_ERR_UNSUPPORTED;
    if (!cu_q_lens && total_q_tokens != num_seqs) return KV_ERR_INVALID;
    if (!(scale > 0.f) || !std::isfinite(scale)) return KV_ERR_INVALID;
    if (!pkv_host::aligned(out, 16) || !pkv_host::aligned(q, 16) || !pkv_host::aligned(cache, 16) ||
        !pkv_host::aligned(block_tables, 4) || !pkv_host::aligned(context_lens, 4) ||
        (cu_q_lens && !pkv_host::aligned(cu_q_lens, 4)))
        return KV_ERR_INVALID;
    const size_t need =
        paged_latent_attention_workspace_size(num_seqs, total_q_tokens, num_heads, max_blocks_per_seq);
    if (need && (!workspace || workspace_bytes < need || !pkv_host::aligned(workspace, 256))) return KV_ERR_INVALID;
    const Plan y = plan((int64_t)total_q_tokens * num_heads <= 64ll * num_seqs && num_heads <= 64);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    LatentParams p;
    p.out = static_cast<uint16_t *>(out);
    p.q = static_cast<const uint16_t *>(q);
    p.cu = cu_q_lens;
    p.lens = context_lens;
    p.tables = block_tables;
    p.desc = reinterpret_cast<int4 *>(ws);
    p.desc2 = reinterpret_cast<int64_t *>(ws + y.desc2);
    p.part_ml = reinterpret_cast<float *>(ws + y.ml);
    p.part_o = reinterpret_cast<float *>(ws + y.o);
    p.unit = y.unit;
    p.workers = y.workers;
    p.num_seqs = num_seqs;
    p.rows = total_q_tokens;
    p.heads = num_heads;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * LOG2E;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (y.small) {
        const kv_status launched = pkv_latent_small::launch(&p, q, cache, st);
        if (launched != KV_OK) return launched;
    } else {
        // the cache as rows of 576: boxes of 16 rows (a block) x 64 latent or 32 rotary dims
        CUtensorMap lmap, rmap;
        const uint64_t rows = (uint64_t)num_blocks * BS;
        if (!pkv_host::encode_tmap_2d(&lmap, cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, LKD, rows, LKD * 2, 64, BS,
                                      CU_TENSOR_MAP_SWIZZLE_128B) ||
            !pkv_host::encode_tmap_2d(&rmap, cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, LKD, rows, LKD * 2, RHALF, BS,
                                      CU_TENSOR_MAP_SWIZZLE_64B))
            return KV_ERR_CUDA;
        if (pkv_host::ensure_dynamic_smem<latent_kernel>(SMEM_BYTES) != cudaSuccess) return KV_ERR_CUDA;
        if (pkv_host::launch_ex(latent_kernel, dim3(2 * NCL), dim3(THREADS), SMEM_BYTES, st, true, lmap, rmap, p) != cudaSuccess)
            return KV_ERR_CUDA;
    }
    if (pkv_host::launch_ex(latent_merge_kernel, dim3(MERGE_CTAS), dim3(256), 0, st, true, p) != cudaSuccess) return KV_ERR_CUDA;
    return KV_OK;
}

}  // extern "C"
