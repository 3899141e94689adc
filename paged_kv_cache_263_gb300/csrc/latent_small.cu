// latent_small.cu -- attention over a paged latent cache, absorbed form, for units
// of up to 64 query rows (sm_103a, 5th-generation tensor cores).
//
// The same operator as latent_decode.cu, which see; there, 128 rows take two CTAs.
// With up to 64 (row, head) columns one CTA holds everything if the products are
// turned round, with keys and dims along M and the query columns along N:
//   S^T[64 keys x N] = K Q^T,   O^T[512 x N] += V^T P^T (four products of 128 dims)
// Nothing is exchanged with another CTA, and what a product costs falls with N.
//  * Bound by memory at few columns: a tile of 64 keys is 72 KiB, 3,100 cycles of a
//    SM's share of the bandwidth, and the products take 1,540 (N = 16).  256 sequences
//    of 17 to 4,096 tokens, 8 heads: 117 us, 5.2 TB/s; a tile takes 3,300 cycles, and
//    12,000 of 200,000 go by until the first has landed.
//  * At 64 columns the products take 2,050 cycles, all of them at the full rate of
//    shared memory (128 bytes a cycle: both operands come from there), and the loads'
//    576 come on top: a tile takes 3,700.  One context of 131,072, 64 heads: 47 us, of
//    which the tiles are 25, the way to the first tile 6; the partial sums of 152 CTAs
//    (20 MB out and in again) and the merge take the rest.  (Two such CTAs a 128-row
//    unit, each tile loaded once for both, were 17 % slower than latent_decode.cu for 64
//    sequences x 128 heads.)
//  * Shared memory: queries 72 KiB, two key stages of 72 KiB, P^T 8 KiB.  A stage is
//    the K-major A operand of the first product and the MN-major A operand of the
//    second.
//  * Tensor memory: S^T 2 x 64 columns, O^T 4 x 64, and 64 for the row sums: a
//    product of a block of ones with P^T adds up exactly the bf16 values that the
//    second product uses, and no thread has to.
//  * Softmax: warps w and w + 4 hold keys 16 w .. 16 w + 15 of the tile and half of
//    its columns each, a thread two keys and column pairs.  A column's reference is a
//    power of two near its first scores and moves only when an exponential exceeds
//    2^15 (by a power of two, so without error).  The warps do not wait for each other
//    to learn of that: the issuer of the second products refuses the tile, and it is
//    done again.
//  * A tile is loaded, multiplied and released in two halves of its dims, so that a
//    stage is filled again while its other half is still in use (5 % of the time).
// Warps 0-7: softmax and epilogue; 8: TMA producer; 9: first products; 10: second.
#include "latent_work.cuh"

#include <cmath>

namespace {

constexpr float FAR = 32768.0f;
constexpr float NO_REF = -3.0e38f;                // no score yet: any finite one is far above
constexpr int STAGES = 2;
constexpr uint32_t CHUNK_BYTES = TK * 128;        // 64 keys (or query columns) x 64 dims
constexpr uint32_t TILE_BYTES = 9 * CHUNK_BYTES;  // eight latent chunks and the rotary one
constexpr uint32_t SSTAGE = TILE_BYTES;           // the queries come first
constexpr uint32_t SP = SSTAGE + STAGES * TILE_BYTES, SONES = SP + TK * 128, SBAR = SONES + 1024;
constexpr uint32_t LIST_OFF = 736;                // within the barrier area
constexpr int LIST = 24;
constexpr int SMEM_BYTES = SBAR + 1024;
constexpr int SOFT = 8;                           // softmax warps
constexpr int W_PROD = SOFT, W_S = SOFT + 1, W_PV = SOFT + 2, THREADS = 32 * (SOFT + 3);
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");

enum {
    B_KVF = 0,                  // + 2 stage + half: it landed (latent dims 0-255; the others and the rotary ones)
    B_KVE = B_KVF + 2 * STAGES, // + 2 stage + half: every product that reads it has finished
    B_Q = B_KVE + 2 * STAGES,      // the item's queries landed
    B_QFREE = B_Q + 1,          // every first product of the item has finished
    B_S = B_QFREE + 1,          // + buffer: S^T is in tensor memory
    B_SFREE = B_S + 2,          // + buffer: it is not needed any more (8 warps)
    B_P = B_SFREE + 2,          // P^T is in shared memory (8 arrivals)
    B_PVD = B_P + 1,            // it has been used, or refused
    B_OFREE = B_PVD + 1,        // the item's O^T was read (8 arrivals)
    B_MEET = B_OFREE + 1,       // the softmax warps meet (8 arrivals)
    B_END = B_MEET + 1,         // + issuer: everything it issued has finished
    NBAR = B_END + 2
};
// after the barriers: tensor memory address, abort flag, start[3], votes[2], -, cut[4]; then 64 each of
// the columns' references, key limits and (in turn) sums
constexpr uint32_t REF_OFF = 224;
static_assert(NBAR * 8 + 8 + 24 + 32 <= REF_OFF && REF_OFF + 2 * 256 == LIST_OFF && LIST_OFF + LIST * 12 <= 1024, "barrier area");

constexpr uint32_t idesc(int m, int n, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? (1u << 15) : 0u) | (b_mn ? (1u << 16) : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

// 16 lanes x 32 columns of a warp's quarter of tensor memory: v[j][0..1] row lane / 4,
// columns 8 j + 2 (lane % 4) and the next; v[j][2..3] row lane / 4 + 8
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&v)[4][4])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i >> 2][i & 3] = __uint_as_float(r[i]);
}

__global__ void __launch_bounds__(THREADS, 1)
    latent_small_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap, const LatentParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SBAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NBAR);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *s_start = reinterpret_cast<int *>(tmem_slot + 2);
    volatile int *votes = reinterpret_cast<volatile int *>(tmem_slot + 5);
    int *s_cut = reinterpret_cast<int *>(tmem_slot + 8);
    volatile float *ref_sh = reinterpret_cast<volatile float *>(smem + SBAR + REF_OFF);
    volatile int *lim_sh = reinterpret_cast<volatile int *>(smem + SBAR + REF_OFF + 256);
    int *list = reinterpret_cast<int *>(smem + SBAR + LIST_OFF);
    auto bar = [&](int i) -> uint32_t { return sbase + SBAR + i * 8; };
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int k = blockIdx.x;
    griddep_launch_dependents();
    if (sbase & 1023u) {
        // the 128-byte swizzle needs 1 KiB-aligned tiles (there is no room to align
        // them here; the array starts on such a boundary): refuse rather than
        // compute with a wrong layout
        if (threadIdx.x == 0) flag(ST_TIMEOUT);
        griddep_wait();
        if (threadIdx.x == 0) p.desc[k] = make_int4(0, 0, 0, 0);
        return;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * STAGES; ++i) {
            mbar_init(bar(B_KVF + i), 1);
            mbar_init(bar(B_KVE + i), 1);
        }
        mbar_init(bar(B_Q), 1);
        mbar_init(bar(B_QFREE), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_SFREE + i), SOFT);
            mbar_init(bar(B_END + i), 1);
        }
        mbar_init(bar(B_P), SOFT);
        mbar_init(bar(B_PVD), 1);
        mbar_init(bar(B_OFREE), SOFT);
        mbar_init(bar(B_MEET), SOFT);
        *abort_flag = 0;
        s_start[0] = p.num_seqs;
        s_start[1] = s_start[2] = 0;
        votes[0] = votes[1] = 0;
        fence_mbar_init();
        prefetch_tmap(&qmap);
        prefetch_tmap(&kmap);
    }
    if (warp == W_PROD) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    // an atom of ones, 8 keys x 64 rows (bf16 1.0)
    for (int i = threadIdx.x; i < 64; i += THREADS) st_shared_v4(sbase + SONES + i * 16, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    fence_proxy_async_smem();
    tc_fence_before();
    griddep_wait();       // everything below reads what earlier kernels wrote
    constexpr pkv_split::Rule rule = pkv_split::ONE;
    const Range range = find_range<THREADS>(p, rule, k, k == 0, reinterpret_cast<int *>(smem + SP), s_start, s_cut, list, LIST);
    Walk walk = {uniform(range.walk.s), uniform(range.walk.u), uniform(range.walk.j), uniform(range.walk.left)};
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    const uint32_t tO = tmem + 128, tL = tmem + 384;              // S^T at 64 b
    Item it = {};
    // columns that the products take: the unit's rows, in steps of 16
    auto columns = [&]() -> int { return (it.rows + 15) & ~15; };

    if (warp == W_PROD) {
        // ======================= producer: a box of 2 KiB (a block's 16 keys x 64 dims)
        // at a time, issued by one elected lane (every 27 cycles; with a lane for each box
        // they left every 70, 2,500 cycles a tile); each lane reads the id of block
        // lane % 4 of the next tile while it waits
        const int blk = lane & 3;
        int u = 0, items = 0, asked = 0;   // halves, items, items whose queries have been asked for
        bool ok = true;
        for (; ok && next_item(p, range, walk, it); ++items) {
            const int32_t *bt = p.tables + (size_t)it.s * p.max_blocks;
            const int nblk = (it.q.L + BS - 1) / BS;
            auto block_id = [&](int j) -> int32_t {
                const int b = j * (TK / BS) + blk;
                return (j < it.j1 && b < nblk) ? __ldg(bt + b) : -1;
            };
            int32_t next_id = block_id(it.j0);
            auto queries = [&]() {
                const int boxes = columns() / 16 * 9;                 // 16 rows x 64 dims each
                if (lane == 0) mbar_arrive_expect_tx(bar(B_Q), boxes * 2048);
                __syncwarp();
                for (int e = lane; e < boxes; e += 32)
                    tma_load_2d(sbase + (e % 9) * CHUNK_BYTES + (e / 9) * 2048, &qmap, (e % 9) * 64,
                                it.q.a * p.heads + it.r0 + (e / 9) * 16, bar(B_Q));
                ++asked;
            };
            if (items == 0) queries();
            for (int j = it.j0; ok && j < it.j1; ++j) {
                const int32_t id = next_id;
                next_id = block_id(j + 1);
                const bool in = j * (TK / BS) + blk < nblk, valid = in && id >= 0 && id < p.num_blocks;
                if (in && !valid && lane < 4) flag(ST_BAD_BLOCK);
                const unsigned vm = __ballot_sync(0xffffffffu, valid) & 15u;
                int32_t rows[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) rows[b] = __shfl_sync(0xffffffffu, id, b) * BS;
                for (int h = 0; h < 2; ++h, ++u) {
                    const int st = (u >> 1) % STAGES, sh = 2 * st + h, turn = (u >> 1) / STAGES;
                    if (turn > 0 && !wait_bar(bar(B_KVE + sh), (turn - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        fence_proxy_async_smem();
                        mbar_arrive_expect_tx(bar(B_KVF + sh), __popc(vm) * (4 + h) * 2048);
                        const uint32_t at = sbase + SSTAGE + st * TILE_BYTES + h * 4 * CHUNK_BYTES;
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            if (!(vm >> b & 1)) continue;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                tma_load_2d(at + e * CHUNK_BYTES + b * 2048, &kmap, (4 * h + e) * 64, rows[b], bar(B_KVF + sh));
                            if (h == 1) tma_load_2d(at + 4 * CHUNK_BYTES + b * 2048, &kmap, LAT, rows[b], bar(B_KVF + sh));
                        }
                    }
                    __syncwarp();
                }
                // the item's queries, once every first product of the item before has finished
                // (rows past the unit's are multiplied along, never stored)
                if (ok && j == it.j0 && items > 0) {
                    ok = wait_bar(bar(B_QFREE), (items - 1) & 1, abort_flag);
                    if (ok) queries();
                }
            }
        }
        if (*abort_flag) {    // loads in flight land before the CTA exits
            for (int x = max(0, u - 2 * STAGES); x < u; ++x)
                (void)mbar_wait_bounded(bar(B_KVF + 2 * ((x >> 1) % STAGES) + (x & 1)), ((x >> 1) / STAGES) & 1);
            if (asked > 0) (void)mbar_wait_bounded(bar(B_Q), (asked - 1) & 1);
        }
    } else if (warp == W_S) {
        // ======================= S^T = K Q^T
        const uint64_t qdesc = sdesc_sw128(sbase, 16, 1024), kdesc = sdesc_sw128(sbase + SSTAGE, 16, 1024);
        int x = 0, items = 0;
        bool ok = true;
        for (; ok && next_item(p, range, walk, it); ++items) {
            const uint32_t id = idesc(64, 0, false, false) | ((uint32_t)(columns() >> 3) << 17);
            ok = wait_bar(bar(B_Q), items & 1, abort_flag);
            for (int j = it.j0; ok && j < it.j1; ++j, ++x) {
                const int st = x % STAGES, b = x & 1;
                if (x >= 2 && !wait_bar(bar(B_SFREE + b), ((x >> 1) - 1) & 1, abort_flag)) { ok = false; break; }
                const int first = it.q.L - j * TK;
                const uint64_t kd = kdesc + (uint64_t)((st * TILE_BYTES) >> 4);
                auto half = [&](int h, int k0, int k1) -> bool {
                    if (!wait_bar(bar(B_KVF + 2 * st + h), (x / STAGES) & 1, abort_flag)) return false;
                    if (first < TK) {
                        // keys at or past the context's end may hold anything (never written, or not
                        // loaded); P is 0 there, but 0 x NaN is NaN
                        const uint32_t vb = sbase + SSTAGE + st * TILE_BYTES + 4 * h * CHUNK_BYTES;
                        for (int e = lane; e < (TK - first) * 32; e += 32)
                            st_shared_v4(vb + ((e >> 3) & 3) * CHUNK_BYTES + (first + (e >> 5)) * 128 + (e & 7) * 16, 0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (elect_one()) {
                        tc_fence_after();
#pragma unroll
                        for (int kk = k0; kk < k1; ++kk)
                            umma_f16(tmem + b * 64, kd + (uint64_t)(((kk >> 2) * CHUNK_BYTES + (kk & 3) * 32) >> 4),
                                     qdesc + (uint64_t)(((kk >> 2) * CHUNK_BYTES + (kk & 3) * 32) >> 4), id, kk > 0);
                        if (h == 1) {
                            umma_commit(bar(B_S + b));
                            if (j == it.j1 - 1) umma_commit(bar(B_QFREE));
                        }
                    }
                    __syncwarp();
                    return true;
                };
                ok = half(0, 0, 16) && half(1, 16, LKD / 16);
            }
        }
        if (elect_one()) umma_commit(bar(B_END));
        __syncwarp();
        (void)mbar_wait_bounded(bar(B_END), 0);
    } else if (warp == W_PV) {
        // ======================= O^T += V^T P^T, and the sums
        const uint64_t vdesc = sdesc_sw128(sbase + SSTAGE, CHUNK_BYTES, 1024), pdesc = sdesc_sw128(sbase + SP, CHUNK_BYTES, 1024);
        const uint64_t ones = sdesc_sw128(sbase + SONES, 16, 0);      // one atom for every group of 8 keys
        int x = 0, items = 0, pn = 0;
        bool ok = true;
        for (; ok && next_item(p, range, walk, it); ++items) {
            const uint32_t n = (uint32_t)(columns() >> 3) << 17;
            const uint32_t idv = idesc(128, 0, true, true) | n, idl = idesc(64, 0, true, true) | n;
            if (items > 0) ok = wait_bar(bar(B_OFREE), (items - 1) & 1, abort_flag);
            for (int j = it.j0; ok && j < it.j1; ++pn) {
                const int st = x % STAGES;
                if (!wait_bar(bar(B_P), pn & 1, abort_flag)) { ok = false; break; }
                const bool refused = votes[pn & 1] == pn + 1;
                if (elect_one()) {
                    if (!refused) {
                        tc_fence_after();
                        const uint64_t vd = vdesc + (uint64_t)((st * TILE_BYTES) >> 4);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
#pragma unroll
                            for (int kk = 0; kk < TK / 16; ++kk)
                                umma_f16(tO + 64 * m, vd + (uint64_t)((2 * m * CHUNK_BYTES + kk * 2048) >> 4),
                                         pdesc + (uint64_t)((kk * 2048) >> 4), idv, (j > it.j0 || kk > 0) ? 1u : 0u);
                            if (m & 1) umma_commit(bar(B_KVE + 2 * st + (m >> 1)));
                        }
#pragma unroll
                        for (int kk = 0; kk < TK / 16; ++kk)
                            umma_f16(tL, ones, pdesc + (uint64_t)((kk * 2048) >> 4), idl, (j > it.j0 || kk > 0) ? 1u : 0u);
                    }
                    umma_commit(bar(B_PVD));
                }
                __syncwarp();
                if (!refused) {
                    ++j;
                    ++x;
                }
            }
        }
        if (elect_one()) umma_commit(bar(B_END + 1));
        __syncwarp();
        (void)mbar_wait_bounded(bar(B_END + 1), 0);
    } else {
        // ======================= softmax and epilogue
        const int w = warp & 3, grp = warp >> 2, tid = threadIdx.x, rw = lane >> 2, cp = 2 * (lane & 3);
        const uint32_t lane_base = (uint32_t)(w * 32) << 16;
        volatile float *scratch = reinterpret_cast<volatile float *>(smem + SP);     // [4][64], then factors [64]: while P^T is not in use
        int x = 0, pn = 0, met = 0;
        const float sl = p.scale_log2;
        bool ok = true, merges = false;
        auto meet = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_MEET));
            return wait_bar(bar(B_MEET), met++ & 1, abort_flag);
        };
        while (ok && next_item(p, range, walk, it)) {
            const int rows = it.rows, N = columns();
            const int c0 = grp * (N >> 1), steps = N >> 4;                      // this warp's columns: 8 steps from c0
            // keys that the first row sees
            const int see0 = it.q.L > 0 ? it.q.L - it.q.n + 1 + (int)((uint32_t)it.r0 / (uint32_t)p.heads) : 0;
            if (tid < 64) {
                lim_sh[tid] = it.q.L > 0 ? it.q.L - it.q.n + 1 + (int)((uint32_t)(it.r0 + min(tid, rows - 1)) / (uint32_t)p.heads) : 0;
                ref_sh[tid] = 0.f;
            }
            if (!meet()) break;
            float nref[4][2];                                                   // minus the references
            for (int j = it.j0;;) {
                bool redo = false;
                if (j > it.j0) {
                    // P^T of the tile before has been used, or refused
                    if (!wait_bar(bar(B_PVD), (pn - 1) & 1, abort_flag)) { ok = false; break; }
                    redo = votes[(pn - 1) & 1] == pn;
                    if (!redo && lane == 0) mbar_arrive(bar(B_SFREE + ((x - 1) & 1)));
                }
                if (!redo) {
                    if (j == it.j1) break;
                    if (!wait_bar(bar(B_S + (x & 1)), (x >> 1) & 1, abort_flag)) { ok = false; break; }
                }
                tc_fence_after();
                const int tj = redo ? j - 1 : j, key0 = tj * TK + w * 16 + rw;  // this thread's keys: key0 and key0 + 8
                const bool masked = (tj + 1) * TK > see0, move = redo || j == it.j0;
                float v[4][4];
                tmem_ld_16x32(tmem + (((redo ? x - 1 : x) & 1) * 64 + c0) + lane_base, v);
                if (masked) {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int lim = lim_sh[(c0 + 8 * h + cp + e) & 63];
                            if (key0 >= lim) v[h][e] = -INFINITY;
                            if (key0 + 8 >= lim) v[h][2 + e] = -INFINITY;
                        }
                }
                if (move) {
                    // the columns' largest scores in this tile
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        if (h >= steps) continue;
                        const int col = c0 + 8 * h + cp;
                        float m0 = fmaxf(v[h][0], v[h][2]), m1 = fmaxf(v[h][1], v[h][3]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) {
                            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
                        }
                        if (rw == 0) {
                            scratch[w * 64 + col] = m0;
                            scratch[w * 64 + col + 1] = m1;
                        }
                    }
                    if (!meet()) { ok = false; break; }
                    if (tid < N) {
                        const float mx = fmaxf(fmaxf(scratch[tid], scratch[64 + tid]), fmaxf(scratch[128 + tid], scratch[192 + tid])) * sl;
                        const float old = ref_sh[tid];
                        const float now = mx == -INFINITY ? (tj == it.j0 ? NO_REF : old) : tj == it.j0 ? ceilf(mx) : fmaxf(old, ceilf(mx));
                        ref_sh[tid] = now;
                        scratch[256 + tid] = ex2(old - now);          // a power of two
                    }
                    if (!meet()) { ok = false; break; }
                    if (redo) {
                        // O^T and the sums, by column
#pragma unroll 1
                        for (int c = 16 * grp; c < 5 * 64; c += 32) {
                            if ((c & 63) >= N) continue;
                            float o[16];
                            tmem_ld16(tO + lane_base + c, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= scratch[256 + (c & 63) + e];
                            tmem_st16(tO + lane_base + c, o);
                        }
                        tmem_wait_st();
                    }
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        nref[h][0] = -ref_sh[(c0 + 8 * h + cp) & 63];
                        nref[h][1] = -ref_sh[(c0 + 8 * h + cp + 1) & 63];
                    }
                    if (!meet()) { ok = false; break; }               // the scratch is P^T's from here on
                }
                float big = 0.f;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if (h >= steps) continue;
                    // raw scores; the scale (> 0) is applied inside the exponent's FFMA
                    const float q0 = ex2(fmaf(v[h][0], sl, nref[h][0])), q1 = ex2(fmaf(v[h][1], sl, nref[h][1]));
                    const float q2 = ex2(fmaf(v[h][2], sl, nref[h][0])), q3 = ex2(fmaf(v[h][3], sl, nref[h][1]));
                    big = max3(big, fmaxf(q0, q1), fmaxf(q2, q3));
                    // P^T as the MN-major operand: a key's 64 columns in 128 bytes, 16-byte pieces
                    // permuted by the key's bits 0-2 (both of a thread's keys have the same)
                    const uint32_t at = sbase + SP + (w * 16 + rw) * 128 + ((((c0 >> 3) + h) ^ rw) << 4) + (lane & 3) * 4;
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(pack_bf16(q0, q1)) : "memory");
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 1024), "r"(pack_bf16(q2, q3)) : "memory");
                }
                // Far above the reference, the tile is refused: its second products are not
                // issued, and it is done again with a reference that has moved.  (fp32 and bf16
                // keep their relative precision whatever the reference, so it moves only to keep
                // clear of overflow.)
                if (!move && __any_sync(0xffffffffu, big > FAR) && lane == 0) votes[pn & 1] = pn + 1;
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_P));
                ++pn;
                if (!redo) {
                    ++j;
                    ++x;
                }
            }
            if (!ok) break;
            tc_fence_after();
            const bool whole = it.whole();
            const int slot = pkv_split::own_slot(k, it);
            const size_t row0 = (size_t)it.q.a * p.heads + it.r0, pr0 = (size_t)slot * p.unit;
            // the sums: every lane of their accumulator holds the column's
            volatile float *sum_sh = reinterpret_cast<volatile float *>(const_cast<int *>(lim_sh));
            if (w == 0) {
                float v[4][4];
                tmem_ld_16x32(tL + c0, v);
                if (rw == 0) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        if (h >= steps) continue;
                        sum_sh[c0 + 8 * h + cp] = v[h][0];
                        sum_sh[c0 + 8 * h + cp + 1] = v[h][1];
                    }
                }
            }
            if (!meet()) break;
            if (tid < rows) {
                const float l = sum_sh[tid];
                if (!whole) {
                    p.part_ml[2 * (pr0 + tid)] = l == 0.f ? -INFINITY : ref_sh[tid];
                    p.part_ml[2 * (pr0 + tid) + 1] = l;
                }
                sum_sh[tid] = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
            }
            if (!meet()) break;
            // a lane holds one dim of 16 columns (rows of the output) at a time
#pragma unroll 1
            for (int c = grp * 128; c < (grp + 1) * 128; c += 16) {
                const int col = c & 63, dim = (c >> 6) * 128 + w * 32 + lane;
                if (col >= N) continue;
                float o[16];
                tmem_ld16(tO + lane_base + c, o);
                if (whole) {
                    // two lanes exchange, so that each stores two dims
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a = o[e] * sum_sh[col + e], z = o[e + 8] * sum_sh[col + e + 8];
                        const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : z, 1);
                        const int row = col + e + (lane & 1) * 8;
                        if (row < rows)
                            *reinterpret_cast<uint32_t *>(p.out + (row0 + row) * LAT + (dim & ~1)) = lane & 1 ? pack_bf16(got, z) : pack_bf16(a, got);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (col + e < rows) p.part_o[(pr0 + col + e) * LAT + dim] = o[e];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_OFREE));
            if (!whole && it.j0 == 0 && tid == 0) {
                list_merge(p, range, it, k, rows);
                merges = true;
            }
            if (!meet()) break;       // the limits and references may be the next item's
        }
        // (the workspace starts with anything)
        if (!merges && tid == 0) p.desc[k] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
    if (warp == W_PROD) tmem_dealloc(tmem, 512);
}

}  // namespace

namespace pkv_latent_small {

cudaError_t status_word(uint32_t **at) { return cudaGetSymbolAddress(reinterpret_cast<void **>(at), g_status); }

// params: a LatentParams with units of 64
kv_status launch(const void *params, const void *q, const void *cache, cudaStream_t st)
{
    const LatentParams &p = *static_cast<const LatentParams *>(params);
    CUtensorMap qmap, kmap;
    if (!pkv_host::encode_tmap_2d(&qmap, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, LKD, (uint64_t)p.rows * p.heads, LKD * 2, 64, 16,
                                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !pkv_host::encode_tmap_2d(&kmap, cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, LKD, (uint64_t)p.num_blocks * BS, LKD * 2, 64, BS,
                                  CU_TENSOR_MAP_SWIZZLE_128B))
        return KV_ERR_CUDA;
    if (pkv_host::ensure_dynamic_smem<latent_small_kernel>(SMEM_BYTES) != cudaSuccess) return KV_ERR_CUDA;
    return pkv_host::launch_ex(latent_small_kernel, dim3(p.workers), dim3(THREADS), SMEM_BYTES, st, true, qmap, kmap, p) == cudaSuccess
               ? KV_OK : KV_ERR_CUDA;
}

}  // namespace pkv_latent_small
