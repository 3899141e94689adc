// latent_prefill.cu -- attention over expanded latents, for prompts (sm_103a,
// 5th-generation tensor cores).
//
// kv[t][h] holds head h's key part (128, expanded from the token's latent) and
// value (128); the rotary key k_rope[t] (64) is shared by all heads:
//   out[r][h] = sum_t p_t kv[t][h][128:],
//   p = softmax_t(scale * (q[r][h][:128] . kv[t][h][:128] + q[r][h][128:] . k_rope[t]))
// over the keys t <= nk - nq + i that row i of a sequence's nq rows sees.
//
// What bounds it: 2 x 320 operations a (row, head, key) on the tensor cores.  A
// work item is one head's 256 query rows (a pair of 128-row tiles) of a sequence
// with every key they see, so a key tile that was loaded serves 256 rows.
//  * Key tiles of 128, in chunks of 128 keys x 64 dims (16 KiB, one TMA box each):
//    the key part's two, the rotary one, the value's two -- read in place from kv
//    and k_rope.  Eight chunks circulate in a ring beside the queries (96 KiB).
//  * S[128 x 128] = Q K^T (A and B in shared memory) and O[128 x 128] += P V (A =
//    P in bf16, written over S) run as tcgen05.mma.  128 keys a tile because a
//    128 x 64 x 16 product with A in shared memory takes 48 cycles and a 128 x 128
//    x 16 one 65 (measured): the query tile is read once per product.
//  * Tensor memory holds one S and one O of each query tile: 512 columns.  The two
//    tiles take turns: while one's softmax works, the other's products run, so the
//    softmax has to be as quick as they are (1,300 cycles).  It takes its reference
//    maximum from the first key tile and keeps it: a later tile's exponentials are
//    computed at once, and only if their sum shows a score far above the reference
//    is the maximum taken, the output rescaled and the tile done again.
//  * One CTA a SM takes items from a list, a device-built one: sequences with the
//    most keys first, within a sequence eight heads at a time (their keys stay in
//    L2 while all their query tiles pass), longest tiles first.
//  * Each query tile goes on to its next item by itself: its queries are loaded as
//    soon as its own first products are through, and its first product runs beside
//    the other tile's last ones.  (Waiting for each other cost 4,000 cycles an item:
//    442 us for 4,096 tokens x 128 heads in a short run, 435 without.)
//  * What is left: both operands of S come from shared memory at its full rate, 128
//    bytes a cycle, and the loads' writes and P V's reads share it -- 168 KiB, 1,310
//    cycles of a 1,770-cycle turn.  Handing P on in halves, so that P V starts before
//    the softmax ends, changes nothing in that.
//    4,096 tokens x 128 heads: 477 us in a long run, at the clock that the power limit
//    leaves (1.44 PFLOP/s), 438 in a short one; six chunks of 333 to 2,048 tokens over
//    799 to 2,398 keys, 64 heads: 278 and 260 us; eight of 40 to 300 tokens, 32 heads:
//    21 us.
//  * The sum that a row is divided by adds its probabilities as fp32, before their
//    rounding to bf16 for the second product.  Adding the rounded ones would cancel
//    part of the rounding (see latent_decode.cu) and costs 2.5 % (a mixed addition for
//    each instead of one a pair, 437 to 448 us; 459 with integer operations to unpack
//    them, 464 once P has been handed on, for the registers that it then holds).
// Warps 0 and 1: MMA issuers of the query tiles, which take turns; 2: TMA; 3: items;
// 4-7 and 8-11: softmax and epilogue of the query tiles, one row a thread.
#include "common.cuh"
#include "latent_loads.h"
#include "trace.h"

#include <algorithm>
#include <cmath>

namespace {

__device__ uint32_t g_status;

using namespace pkv;

constexpr float LOG2E = 1.4426950408889634f;
constexpr float FAR = 32768.0f;                  // a tile's sum above this: its maximum is taken anew
constexpr int QKD = D + ROPE;                     // 192
constexpr int BM = 128, BN = 128, PAIR = 2 * BM;
constexpr int HGROUP = 8;                         // heads whose items are adjacent
constexpr int CHUNKS = 8;
constexpr uint32_t CHUNK_BYTES = BN * 128, Q_TILE = 3 * BM * 128;
constexpr uint32_t SKV = 2 * Q_TILE, SBAR = SKV + CHUNKS * CHUNK_BYTES;
constexpr int SMEM_BYTES = SBAR + 512 + 1024;     // + 1 KiB: aligned to 1 KiB at run time
constexpr int W_MMA = 0, W_PROD = 2, W_ITEM = 3, W_SOFT = 4, THREADS = 32 * (W_SOFT + 8);
constexpr int NSLOT = 2;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");

enum {
    B_K0 = 0,                       // + key tile parity: its first key chunk landed
    B_KF = B_K0 + 2,                // + key tile parity: its second key chunk and the rotary one landed
    B_VF = B_KF + 2,                // + key tile parity: its two value chunks landed
    B_KE = B_VF + 2,                // + key tile parity: both its first products have finished (one release an
                                    // issuer; by parity, so that one issuer's releases of two tiles cannot add up)
    B_VE = B_KE + 2,                // + key tile parity: both its second products have finished
    B_TURN = B_VE + 2,              // + query tile: its issuer's turn
    B_Q = B_TURN + 2,               // + query tile: the item's queries landed
    B_QFREE = B_Q + 2,              // + query tile: every first product of the item has finished
    B_S = B_QFREE + 2,              // + tile: S is in tensor memory
    B_P = B_S + 2,                  // + tile: P is (128 arrivals)
    B_DRAIN = B_P + 2,              // + tile: every product of the item has finished
    B_OFREE = B_DRAIN + 2,          // + tile: the item's O was read (128 arrivals)
    B_TAIL = B_OFREE + 2,           // + item parity: value rows past the sequence's end are zeroed (the ring
                                    // lets the producer finish one item ahead, not two)
    B_IFULL = B_TAIL + 2,           // + slot: an item is in the slot
    B_IEMPTY = B_IFULL + NSLOT,     // + slot: every warp has read it
    B_NEXT = B_IEMPTY + NSLOT,      // the item's loads are nearly through: time to take the next
    B_END = B_NEXT + 1,             // + query tile: everything its issuer issued has finished
    NBAR = B_END + 2
};
// an item as the producer hands it on: valid, first query row, rows (up to 256),
// the keys that row 0 sees, first key row, keys of the sequence, head, key tiles
struct Slot {
    int valid, row0, rows, see0, key0, nk, head, T;
    // key tiles of query tile g: the first one's rows may see fewer (rows that see
    // nothing get one tile, all masked)
    __device__ __forceinline__ int tiles(int g) const
    {
        return g == 0 ? max(1, (see0 + min(rows, BM) - 1 + BN - 1) / BN) : T;
    }
};
static_assert(NBAR * 8 + 16 + NSLOT * sizeof(Slot) <= 512, "barrier area");

// instruction descriptors, kind::f16: bf16 A and B, fp32 accumulate, M = 128
constexpr uint32_t idesc(int n, bool b_mn_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn_major ? (1u << 16) : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(BM >> 4) << 24);
}
constexpr uint32_t IDESC_S = idesc(BN, false), IDESC_PV = idesc(64, true);

struct ExpandedParams {
    uint16_t *out;
    const int32_t *cu_q, *cu_k;
    int4 *seqs;          // [num_seqs] sequences by falling key count: first row, rows, first key, keys
    int32_t *before;     // [num_seqs + 1] items of the sequences before
    int32_t *next;       // the next item that no CTA has taken
    int num_seqs, rows, keys, heads;
    int grid, max_items; // CTAs of the attention kernel; items at most
    int small;           // no list: up to 32 sequences, few items (see expanded_kernel)
    float scale_log2;
};

__device__ __forceinline__ void flag(uint32_t bits) { atomicOr(&g_status, bits); }

// The item list: valid sequences with rows, by falling key count (in steps of a
// quarter octave), and the prefix sums of their items.
constexpr int BUCKETS = 128;
__global__ void __launch_bounds__(1024) expanded_plan_kernel(const ExpandedParams p)
{
    __shared__ int count[BUCKETS], start[BUCKETS], total;
    __shared__ long long warp_sum[32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (threadIdx.x < BUCKETS) count[threadIdx.x] = 0;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    auto load = [&](int s, bool flagging) -> int4 {
        const int a = p.cu_q[s], b = p.cu_q[s + 1], c = p.cu_k[s], d = p.cu_k[s + 1];
        if (a == b) return make_int4(0, 0, 0, 0);
        if (a < 0 || b < a || b > p.rows || c < 0 || d < c || d > p.keys) {
            if (flagging) flag(ST_BAD_LEN);
            return make_int4(0, 0, 0, 0);
        }
        return make_int4(a, b - a, c, d - c);
    };
    auto bucket = [](int nk) -> int {
        const int t = (nk >> 5) + 1, e = 31 - __clz(t);                 // quarter octaves of 32 keys
        return BUCKETS - 1 - min(BUCKETS - 1, 4 * e + (e >= 2 ? (t >> (e - 2)) & 3 : 0));
    };
    for (int s = threadIdx.x; s < p.num_seqs; s += 1024) {
        const int4 q = load(s, true);
        if (q.y > 0) atomicAdd(&count[bucket(q.w)], 1);
    }
    __syncthreads();
    if (w == 0) {
        int run = 0;
        for (int b = lane; b < BUCKETS; b += 32) {
            int v = count[b];
            const int n = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += t;
            }
            start[b] = run + v - n;
            run += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) total = run;
    }
    __syncthreads();
    for (int s = threadIdx.x; s < p.num_seqs; s += 1024) {
        const int4 q = load(s, false);
        if (q.y > 0) p.seqs[atomicAdd(&start[bucket(q.w)], 1)] = q;     // (their order within a bucket changes no result)
    }
    __syncthreads();
    const int n = total;
    // (offsets that go backwards could list more items than the caller's sizes
    // allow; what is past that bound is left out)
    long long carry = 0;
    for (int b = 0; b < n; b += 1024) {
        const int i = b + threadIdx.x;
        const long long mine = i < n ? (long long)((p.seqs[i].y + PAIR - 1) / PAIR) * p.heads : 0;
        long long v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
        }
        __syncthreads();
        if (lane == 31) warp_sum[w] = v;
        __syncthreads();
        long long before = carry;
        for (int k = 0; k < 32; ++k) {
            if (k < w) before += warp_sum[k];
            carry += warp_sum[k];
        }
        if (i < n) p.before[i] = (int)min(before + v - mine, (long long)p.max_items);
    }
    if (carry > p.max_items && threadIdx.x == 0) flag(ST_BAD_LEN);
    if (threadIdx.x == 0) {
        p.next[0] = p.grid;           // (its CTAs start with item blockIdx.x)
        p.next[1] = n;
        p.before[n] = (int)min(carry, (long long)p.max_items);
    }
}

// bounded wait that also gives up once another warp of the CTA has.  The loop is a
// call: a dozen copies of it in a role's loop would crowd the instruction cache
__device__ __noinline__ bool wait_loop(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    const unsigned long long t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort_flag) return false;
            if (globaltimer() - t0 > WAIT_LIMIT_NS) {
                *abort_flag = 1;
                flag(ST_TIMEOUT);
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    // (the roles run warp-collective instructions: a warp leaves as a whole)
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || wait_loop(bar, parity, abort_flag));
}

// a box of a tensor into L2
__device__ __forceinline__ void prefetch_tile(const CUtensorMap *map, int32_t x, int32_t y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y)
                 : "memory");
}

__global__ void __launch_bounds__(THREADS, 1)
    expanded_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kvmap,
                    const __grid_constant__ CUtensorMap rmap, const ExpandedParams p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SBAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NBAR);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile Slot *slots = reinterpret_cast<volatile Slot *>(bars + NBAR + 2);
    auto bar = [&](int i) -> uint32_t { return sbase + SBAR + i * 8; };
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_K0 + i), 1);
            mbar_init(bar(B_KF + i), 1);
            mbar_init(bar(B_VF + i), 1);
            mbar_init(bar(B_TURN + i), 1);
            mbar_init(bar(B_END + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_KE + i), 2);
            mbar_init(bar(B_VE + i), 2);
        }
        mbar_init(bar(B_NEXT), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_Q + i), 1);
            mbar_init(bar(B_QFREE + i), 1);
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_P + i), 128);
            mbar_init(bar(B_DRAIN + i), 1);
            mbar_init(bar(B_OFREE + i), 128);
        }
        mbar_init(bar(B_TAIL), 1);
        mbar_init(bar(B_TAIL + 1), 1);
        for (int i = 0; i < NSLOT; ++i) {
            mbar_init(bar(B_IFULL + i), 1);
            mbar_init(bar(B_IEMPTY + i), 11);            // every warp but W_ITEM
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&qmap);
        prefetch_tmap(&kvmap);
        prefetch_tmap(&rmap);
    }
    if (warp == W_PROD) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    // tensor memory: S of tile g at 128 g (P over its first 64 columns), O at 256 + 128 g
    int k = 0;          // items
    // the next item, as every warp but W_ITEM reads it
    auto read_item = [&](Slot &it) -> bool {
        const int sl = k % NSLOT;
        if (!wait_bar(bar(B_IFULL + sl), (k / NSLOT) & 1, abort_flag)) return false;
        it.valid = uniform(slots[sl].valid);
        it.row0 = uniform(slots[sl].row0);
        it.rows = uniform(slots[sl].rows);
        it.see0 = uniform(slots[sl].see0);
        it.key0 = uniform(slots[sl].key0);
        it.nk = uniform(slots[sl].nk);
        it.head = uniform(slots[sl].head);
        it.T = uniform(slots[sl].T);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_IEMPTY + sl));
        return it.valid != 0;
    };
    Slot it;

    if (warp == W_ITEM) {
        // ======================= items
        griddep_wait();                  // the list, and everything before it on the stream
        // small batches (up to 32 sequences, 4 items a CTA) need no list: a lane holds a
        // sequence, and the CTAs take every grid-th item.  That saves the list's
        // kernel, 4 us of the 26 that eight short prompts over 32 heads took
        int ns = 0, items = 0, my_before = INT_MAX;
        int4 mine = make_int4(0, 0, 0, 0);
        if (p.small) {
            if (lane < p.num_seqs) {
                const int a = p.cu_q[lane], b = p.cu_q[lane + 1], c = p.cu_k[lane], d = p.cu_k[lane + 1];
                if (a != b) {
                    if (a < 0 || b < a || b > p.rows || c < 0 || d < c || d > p.keys) {
                        if (blockIdx.x == 0) flag(ST_BAD_LEN);
                    } else {
                        mine = make_int4(a, b - a, c, d - c);
                    }
                }
            }
            // longest first: lane r takes the sequence of rank r (those without rows last)
            const int key = mine.y > 0 ? mine.w : -1;
            int rank = 0, from = 0;
            for (int i = 0; i < 32; ++i) {
                const int other = __shfl_sync(0xffffffffu, key, i);
                rank += other > key || (other == key && i < lane);
            }
            for (int i = 0; i < 32; ++i) {
                const unsigned who = __ballot_sync(0xffffffffu, rank == i);
                if (lane == i) from = __ffs(who) - 1;
            }
            mine = make_int4(__shfl_sync(0xffffffffu, mine.x, from), __shfl_sync(0xffffffffu, mine.y, from),
                             __shfl_sync(0xffffffffu, mine.z, from), __shfl_sync(0xffffffffu, mine.w, from));
            const int n = (mine.y + PAIR - 1) / PAIR * p.heads;      // (offsets are within max_items: checked below)
            long long v = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += x;
            }
            const long long all = __shfl_sync(0xffffffffu, v, 31);
            if (all > p.max_items && lane == 0 && blockIdx.x == 0) flag(ST_BAD_LEN);
            items = (int)min(all, (long long)p.max_items);
            my_before = (int)min(v - n, (long long)p.max_items);
        } else {
            ns = p.next[1];
            items = p.before[ns];
        }
        int idx = blockIdx.x;
        for (;; ++k) {
            const int sl = k % NSLOT;
            if (k >= NSLOT && !wait_bar(bar(B_IEMPTY + sl), (k / NSLOT - 1) & 1, abort_flag)) break;
            if (k > 0) {
                // (not earlier, or an item would wait here that an idle CTA could take)
                if (!wait_bar(bar(B_NEXT), (k - 1) & 1, abort_flag)) break;
                if (p.small) {
                    idx += gridDim.x;
                } else {
                    if (lane == 0) idx = atomicAdd(p.next, 1);
                    idx = __shfl_sync(0xffffffffu, idx, 0);
                }
            }
            it.valid = idx < items;
            if (it.valid) {
                // its sequence: the last one with before <= idx, 32 probes at a time
                int lo = 0, len = ns;
                while (!p.small && len > 1) {
                    const int step = (len + 31) / 32, x = lo + lane * step;
                    const bool le = lane * step < len && p.before[x] <= idx;
                    const int last = 31 - __clz(__ballot_sync(0xffffffffu, le));   // (lane 0 always is)
                    lo += last * step;
                    len = min(step, len - last * step);
                }
                int4 q;
                int r;
                if (p.small) {
                    lo = 31 - __clz(__ballot_sync(0xffffffffu, my_before <= idx && mine.y > 0));   // (lane 0 always is)
                    q = make_int4(__shfl_sync(0xffffffffu, mine.x, lo), __shfl_sync(0xffffffffu, mine.y, lo),
                                  __shfl_sync(0xffffffffu, mine.z, lo), __shfl_sync(0xffffffffu, mine.w, lo));
                    r = idx - __shfl_sync(0xffffffffu, my_before, lo);
                } else {
                    q = p.seqs[lo];
                    r = idx - p.before[lo];
                }
                const int units = (q.y + PAIR - 1) / PAIR;
                const int g0 = r / (units * HGROUP) * HGROUP, gn = min(HGROUP, p.heads - g0);
                const int r2 = r - g0 * units, unit = units - 1 - r2 / gn;
                it.head = g0 + r2 % gn;
                it.row0 = q.x + unit * PAIR;
                it.rows = min(PAIR, q.y - unit * PAIR);
                it.see0 = q.w - q.y + unit * PAIR + 1;
                it.key0 = q.z;
                it.nk = q.w;
                // (rows that see nothing get one tile, all masked)
                it.T = max(1, (it.see0 + it.rows - 1 + BN - 1) / BN);
            }
            if (lane == 0) {
                slots[sl].valid = it.valid;
                slots[sl].row0 = it.row0;
                slots[sl].rows = it.rows;
                slots[sl].see0 = it.see0;
                slots[sl].key0 = it.key0;
                slots[sl].nk = it.nk;
                slots[sl].head = it.head;
                slots[sl].T = it.T;
                mbar_arrive(bar(B_IFULL + sl));
            }
            __syncwarp();
            if (!it.valid) break;
            // its queries' and first keys' way from memory is long: into L2 with them
            if (lane < 9) {
                if (lane >= 6 || it.rows > BM * (lane / 3))
                    prefetch_tile(lane < 6 ? &qmap : lane < 8 ? &kvmap : &rmap,
                                  lane < 6 ? it.head * QKD + 64 * (lane % 3) : lane < 8 ? it.head * 2 * D + 64 * (lane - 6) : 0,
                                  lane < 6 ? it.row0 + BM * (lane / 3) : it.key0);
            }
            __syncwarp();
        }
    } else if (warp == W_PROD) {
        // ======================= loads
        griddep_wait();                  // everything before the kernel on the stream
        int t = 0;                       // key tiles
        bool ok = true;
        pkv_loads::Asked asked;
        int tail_first = BN;             // rows of the last tile loaded that are its sequence's
        auto zero_tail = [&]() -> bool {
            const int x = t - 1, first = max(0, tail_first);
            if (!wait_bar(bar(B_VF + (x & 1)), (x >> 1) & 1, abort_flag)) return false;
            for (int i = 3; i < 5; ++i) {
                const uint32_t vt = sbase + SKV + (uint32_t)((5 * x + i) % CHUNKS) * CHUNK_BYTES;
                for (int e = lane; e < (BN - first) * 8; e += 32) st_shared_v4(vt + (first + (e >> 3)) * 128 + (e & 7) * 16, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_TAIL + ((k - 1) & 1)));
            return true;
        };
        auto queries = [&](int g) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(B_Q + g), Q_TILE);
                for (int i = 0; i < 3; ++i)
                    tma_load_2d(sbase + g * Q_TILE + i * CHUNK_BYTES, &qmap, it.head * QKD + 64 * i, it.row0 + g * BM, bar(B_Q + g));
            }
            ++asked.queries[g];
            __syncwarp();
        };
        for (; ok && read_item(it); ++k) {
            // query tile 0, once every first product of the item before's has finished
            if (k > 0 && !wait_bar(bar(B_QFREE), (k - 1) & 1, abort_flag)) break;
            queries(0);
            if (tail_first < BN) {
                // the last tile of the item before holds rows past the sequence's end, of
                // another sequence or of none: P is 0 there, but 0 x NaN is NaN, so their
                // values are zeroed once they have landed (the second product waits for it)
                if (!zero_tail()) break;
            }
            // chunk i of tile t (0, 1 key part, 2 rotary key, 3, 4 value) takes ring slot
            // (5 t + i) % 8, whose last holder was chunk i + 2 of tile t - 2 or i - 3 of t - 1
            for (int j = 0; j < it.T; ++j, ++t) {
                const int y = it.key0 + j * BN;
                auto load = [&](int i, uint32_t b) {
                    const uint32_t dst = sbase + SKV + (uint32_t)((5 * t + i) % CHUNKS) * CHUNK_BYTES;
                    if (i == 2) tma_load_2d(dst, &rmap, 0, y, b);
                    else tma_load_2d(dst, &kvmap, it.head * 2 * D + (i < 2 ? i : i - 1) * 64, y, b);
                };
                const uint32_t k0 = bar(B_K0 + (t & 1)), kb = bar(B_KF + (t & 1)), vb = bar(B_VF + (t & 1));
                // (chunk 0: the keys of tile t - 2 were waited for with the values of t - 1)
                if (lane == 0) {
                    fence_proxy_async_smem();
                    mbar_arrive_expect_tx(k0, CHUNK_BYTES);
                    load(0, k0);
                }
                asked.tiles[pkv_loads::KEY0] = t + 1;
                if (t >= 2 && !wait_bar(bar(B_VE + (t & 1)), ((t - 2) >> 1) & 1, abort_flag)) ok = false;
                if (lane == 0 && ok) {
                    mbar_arrive_expect_tx(kb, 2 * CHUNK_BYTES);
                    load(1, kb);
                    load(2, kb);
                }
                if (ok) asked.tiles[pkv_loads::KEYS] = t + 1;
                if (t >= 1 && ok && !wait_bar(bar(B_KE + ((t - 1) & 1)), ((t - 1) >> 1) & 1, abort_flag)) ok = false;
                if (ok && j == 0) {
                    // query tile 1: its first products of the item before are among those just waited for
                    if (k > 0) ok = wait_bar(bar(B_QFREE + 1), (k - 1) & 1, abort_flag);
                    if (ok && it.rows > BM) {
                        queries(1);
                    } else if (ok) {
                        if (lane == 0) mbar_arrive(bar(B_Q + 1));
                        ++asked.queries[1];
                    }
                }
                if (!ok) break;
                if (lane == 0 && j == max(0, it.T - 3)) mbar_arrive(bar(B_NEXT));
                if (lane == 0) {
                    mbar_arrive_expect_tx(vb, 2 * CHUNK_BYTES);
                    load(3, vb);
                    load(4, vb);
                }
                asked.tiles[pkv_loads::VALUES] = t + 1;
                __syncwarp();
            }
            tail_first = it.nk - (it.T - 1) * BN;
        }
        if (ok && tail_first < BN) (void)zero_tail();
        if (*abort_flag)                 // loads in flight land before the CTA exits
            asked.drain(
                [&](int part, int x) {
                    const int b = part == pkv_loads::KEY0 ? B_K0 : part == pkv_loads::KEYS ? B_KF : B_VF;
                    (void)mbar_wait_bounded(bar(b + (x & 1)), (x >> 1) & 1);
                },
                [&](int g, int x) { (void)mbar_wait_bounded(bar(B_Q + g), x & 1); });
    } else if (warp < W_MMA + 2) {
        // ======================= MMA issuers.  They take turns: one's second product
        // of tile j and first of j + 1, then the other's, so that one query tile's
        // softmax works while the other's products run.  Left alone the two fall into
        // step -- both wait for the softmax, then both for the tensor cores -- and a
        // key tile takes 5,100 cycles; and one warp for both spends its time on
        // barriers (5,300).
        const int g = warp - W_MMA;
        const uint64_t qdesc = sdesc_sw128(sbase + g * Q_TILE, 16, 1024), kvdesc = sdesc_sw128(sbase + SKV, 16, 1024);
        const uint32_t tS = tmem + g * 128, tO = tmem + 256 + g * 128;
        auto chunk = [&](int t, int i) -> uint32_t { return (uint32_t)((5 * t + i) % CHUNKS) * CHUNK_BYTES; };
        int t = 0, n = 0, done = 0;      // key tiles; S tiles and items of this query tile
        int turns = 0;                   // turns this issuer has taken
        unsigned tpar = 0;               // parity of the next tail, by item parity
        bool ok = true;
        for (; ok && read_item(it); ++k) {
            const bool both = it.rows > BM, tail = it.nk < it.T * BN;
            // (both issuers wait for every phase of every barrier in turn: a parity
            // cannot be waited for two phases ahead)
            auto wait_tail = [&]() -> bool {
                const bool zeroed = wait_bar(bar(B_TAIL + (k & 1)), (tpar >> (k & 1)) & 1, abort_flag);
                tpar ^= 1u << (k & 1);
                return zeroed;
            };
            // a tile that this query tile has no use for is released as it lands
            auto pass_by = [&](bool last) -> bool {
                if (!wait_bar(bar(B_K0 + (t & 1)), (t >> 1) & 1, abort_flag) || !wait_bar(bar(B_KF + (t & 1)), (t >> 1) & 1, abort_flag))
                    return false;
                if (lane == 0) mbar_arrive(bar(B_KE + (t & 1)));
                if (!wait_bar(bar(B_VF + (t & 1)), (t >> 1) & 1, abort_flag) || (tail && last && !wait_tail())) return false;
                if (lane == 0) mbar_arrive(bar(B_VE + (t & 1)));
                return true;
            };
            if (g == 1 && !both) {
                ok = wait_bar(bar(B_Q + 1), k & 1, abort_flag);
                if (lane == 0) mbar_arrive(bar(B_QFREE + 1));
                for (int j = 0; ok && j < it.T; ++j, ++t) ok = pass_by(j + 1 == it.T);
                continue;
            }
            const int T = it.tiles(g);
            // the first turn of all is query tile 0's
            auto take_turn = [&]() -> bool {
                if (!both) return true;
                const int x = turns++;
                if (g == 0) return x == 0 || wait_bar(bar(B_TURN), (x - 1) & 1, abort_flag);
                return wait_bar(bar(B_TURN + 1), x & 1, abort_flag);
            };
            // S = Q K^T of key tile x.  Its first chunk is waited for, and multiplied,
            // before the others: those two take the slots of the values before, which
            // the other issuer's products have only just released
            auto issue_s = [&](int x, bool pass, bool last) -> bool {
                auto products = [&](int i) {
                    const uint64_t kd = kvdesc + (uint64_t)(chunk(x, i) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16(tS, qdesc + (uint64_t)((i * CHUNK_BYTES + kk * 32) >> 4), kd + (uint64_t)((kk * 32) >> 4),
                                 IDESC_S, i + kk > 0);
                };
                if (!wait_bar(bar(B_K0 + (x & 1)), (x >> 1) & 1, abort_flag)) return false;
                if (elect_one()) {
                    tc_fence_after();
                    products(0);
                }
                __syncwarp();
                if (!wait_bar(bar(B_KF + (x & 1)), (x >> 1) & 1, abort_flag)) return false;
                if (elect_one()) {
                    tc_fence_after();
                    products(1);
                    // (the turn takes about as long to pass as the last four products)
                    if (pass) mbar_arrive(bar(B_TURN + (g ^ 1)));
                    products(2);
                    umma_commit(bar(B_S + g));
                    umma_commit(bar(B_KE + (x & 1)));
                    if (last) umma_commit(bar(B_QFREE + g));
                }
                __syncwarp();
                return true;
            };
            // (the item's first product takes no turn: it runs beside the other's last ones)
            ok = wait_bar(bar(B_Q + g), k & 1, abort_flag) && issue_s(t, false, T == 1);
            for (int j = 0; ok && j < T; ++j, ++t, ++n) {
                const bool more = j + 1 < T;
                ok = wait_bar(bar(B_VF + (t & 1)), (t >> 1) & 1, abort_flag);
                if (ok && tail && j + 1 == it.T) ok = wait_tail();
                if (ok && j == 0 && done > 0) ok = wait_bar(bar(B_OFREE + g), (done - 1) & 1, abort_flag);
                ok = ok && wait_bar(bar(B_P + g), n & 1, abort_flag) && take_turn();
                if (ok && elect_one()) {
                    tc_fence_after();
                    // O += P V
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            umma_f16_ts(tO + 64 * i, tS + kk * 8,
                                        kvdesc + (uint64_t)((chunk(t, 3 + i) + kk * 2048) >> 4), IDESC_PV, (j > 0 || kk > 0) ? 1u : 0u);
                    umma_commit(bar(B_VE + (t & 1)));
                    if (!more) {
                        umma_commit(bar(B_DRAIN + g));
                        if (both) mbar_arrive(bar(B_TURN + (g ^ 1)));
                    }
                }
                __syncwarp();
                // (in issue order: the products above read P from the columns that S overwrites)
                if (ok && more) ok = issue_s(t + 1, both, j + 2 == T);
            }
            for (int j = T; ok && j < it.T; ++j, ++t) {
                ok = take_turn();
                if (ok && lane == 0) mbar_arrive(bar(B_TURN + (g ^ 1)));
                ok = ok && pass_by(j + 1 == it.T);
            }
            ++done;
        }
        // everything issued has finished before tensor memory is released
        if (elect_one()) umma_commit(bar(B_END + g));
        __syncwarp();
        (void)mbar_wait_bounded(bar(B_END + g), 0);
    } else if (warp >= W_SOFT) {
        // ======================= softmax and epilogue: thread = query row = lane
        const int g = (warp - W_SOFT) >> 2, w = warp & 3, r = threadIdx.x & 127;
        const uint32_t lane_base = (uint32_t)(w * 32) << 16;
        const uint32_t tS = tmem + g * 128 + lane_base, tO = tmem + 256 + g * 128 + lane_base;
        int n = 0, done = 0;             // S tiles and items of this query tile
        const float sl = p.scale_log2;
        bool ok = true;
        for (; ok && read_item(it); ++k) {
            if (g == 1 && it.rows <= BM) continue;
            const int rows = min(BM, it.rows - g * BM);
            // keys that this row sees (rows past the tile's last take the last one's)
            const int see = it.see0 + g * BM + min(r, rows - 1), see_min = it.see0 + g * BM;
            float m_ref = -INFINITY, l = 0.f;
            const int T = it.tiles(g);
            for (int j = 0; j < T; ++j, ++n) {
                if (!wait_bar(bar(B_S + g), n & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const int t0 = j * BN;
                const bool masked = t0 + BN > see_min;
                // 32 raw scores (the scale, > 0, is applied inside the exponent's FFMA)
                auto scores = [&](int c, float (&sv)[32]) {
                    tmem_ld32(tS + 32 * c, sv);
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (t0 + 32 * c + e >= see) sv[e] = -INFINITY;
                    }
                };
                uint32_t pw[BN / 2];
                float sum;
                auto exponentials = [&]() {
                    const float mneg = m_ref == -INFINITY ? 0.f : -m_ref;
                    const uint64_t sl2 = f2_pack(sl, sl), mn2 = f2_pack(mneg, mneg);
                    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float sv[32];
                        scores(c, sv);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float y0, y1;
                            f2_unpack(f2_fma(f2_pack(sv[2 * e], sv[2 * e + 1]), sl2, mn2), y0, y1);
                            const float p0 = ex2(y0), p1 = ex2(y1);
                            acc[e & 3] = f2_add(acc[e & 3], f2_pack(p0, p1));
                            pw[16 * c + e] = pack_bf16(p0, p1);   // the second product's operand type, beside bf16 values
                        }
                    }
                    float s0, s1;
                    f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
                    sum = s0 + s1;
                };
                // P relative to a maximum that is not the largest any more is as exact (fp32
                // and bf16 keep their relative precision) while nothing comes near overflow
                bool fresh = __any_sync(0xffffffffu, m_ref == -INFINITY);
                if (!fresh) {
                    exponentials();
                    fresh = __any_sync(0xffffffffu, sum > FAR);
                }
                if (fresh) {
                    float mk[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float sv[32];
                        scores(c, sv);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
#pragma unroll
                            for (int f = 0; f < 4; ++f) mk[f] = max3(mk[f], sv[e + f], sv[e + 4 + f]);
                    }
                    const float mx = fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])) * sl;
                    const float m_new = fmaxf(m_ref, mx), alpha = m_ref == -INFINITY ? 0.f : ex2(m_ref - m_new);
                    // S(j) was issued after PV(j - 1) and has finished, so PV(j - 1) has
                    if (j > 0) {
#pragma unroll 1
                        for (int h = 0; h < D / 16; ++h) {
                            float o[16];
                            tmem_ld16(tO + h * 16, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= alpha;
                            tmem_st16(tO + h * 16, o);
                        }
                    }
                    l *= alpha;
                    m_ref = m_new;
                    exponentials();
                }
                l += sum;
                tmem_st32u(tS, *reinterpret_cast<const uint32_t(*)[32]>(pw));
                tmem_st32u(tS + 32, *reinterpret_cast<const uint32_t(*)[32]>(pw + 32));
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(B_P + g));
            }
            if (!ok || !wait_bar(bar(B_DRAIN + g), done & 1, abort_flag)) break;
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int r4 = w * 32 + (lane & ~3), e4 = lane & 3;
            uint16_t *dst = p.out + ((size_t)(it.row0 + g * BM) * p.heads + it.head) * D;
#pragma unroll 1
            for (int h = 0; h < D / 32; ++h) {
                float o[32];
                tmem_ld32(tO + h * 32, o);
                // 4 lanes exchange pieces, so that they store 64 bytes of one row together
                uint32_t v[4][4];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e >> 2][e & 3] = pack_bf16(o[2 * e] * inv, o[2 * e + 1] * inv);
                quad_transpose(v, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r4 + i < rows)
                        reinterpret_cast<uint4 *>(dst + (size_t)(r4 + i) * p.heads * D + h * 32)[e4] =
                            make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
            }
            tc_fence_before();
            mbar_arrive(bar(B_OFREE + g));
            ++done;
        }
    }
    __syncthreads();
    if (warp == W_PROD) tmem_dealloc(tmem, 512);
}

// workspace: the sequences, their prefix sums, two counters
struct Layout {
    size_t before, next, total;
};
Layout layout(int num_seqs)
{
    Layout y;
    y.before = ((size_t)num_seqs * sizeof(int4) + 255) & ~(size_t)255;
    y.next = y.before + (((size_t)num_seqs + 1) * 4 + 255 & ~(size_t)255);
    y.total = y.next + 256;
    return y;
}

}  // namespace

namespace pkv_latent_prefill {
cudaError_t status_word(uint32_t **at) { return cudaGetSymbolAddress(reinterpret_cast<void **>(at), g_status); }
}  // namespace pkv_latent_prefill

extern "C" {

size_t latent_prefill_attention_workspace_size(int32_t num_seqs, int32_t total_q_tokens, int32_t num_heads)
{
    if (num_seqs < 1 || total_q_tokens < 1 || num_heads < 1 || num_heads > PAGEDKV_LATENT_MAX_HEADS) return 0;
    return layout(num_seqs).total;
}

kv_status latent_prefill_attention(void *out, const void *q, const void *kv, const void *k_rope,
                                   int64_t k_rope_stride, const int32_t *cu_q_lens, const int32_t *cu_k_lens,
                                   int32_t num_seqs, int32_t total_q_tokens, int32_t total_k_tokens,
                                   int32_t num_heads, float scale, void *workspace, size_t workspace_bytes,
                                   void *stream)
{
    PKV_NVTX_RANGE("latent_prefill_attention");
    if (num_seqs < 0 || total_q_tokens < 0 || total_k_tokens < 0) return KV_ERR_INVALID;
    if (num_seqs == 0 || total_q_tokens == 0) return KV_OK;
    if (num_heads < 1) return KV_ERR_INVALID;
    if (num_heads > PAGEDKV_LATENT_MAX_HEADS) return KV_ERR_UNSUPPORTED;
    if (!out || !q || !cu_q_lens || !cu_k_lens) return KV_ERR_INVALID;
    if (total_k_tokens > 0 && (!kv || !k_rope)) return KV_ERR_INVALID;
    if (!(scale > 0.f) || !std::isfinite(scale)) return KV_ERR_INVALID;
    if (k_rope_stride < ROPE || k_rope_stride % 8) return KV_ERR_INVALID;
    if (!pkv_host::aligned(out, 16) || !pkv_host::aligned(q, 16) || !pkv_host::aligned(kv, 16) ||
        !pkv_host::aligned(k_rope, 16) || !pkv_host::aligned(cu_q_lens, 4) || !pkv_host::aligned(cu_k_lens, 4))
        return KV_ERR_INVALID;
    const size_t need = latent_prefill_attention_workspace_size(num_seqs, total_q_tokens, num_heads);
    if (need && (!workspace || workspace_bytes < need || !pkv_host::aligned(workspace, 256))) return KV_ERR_INVALID;
    // (items are counted in 32 bits)
    const int64_t items = ((int64_t)total_q_tokens / PAIR + num_seqs) * num_heads;
    if (items > INT32_MAX) return KV_ERR_UNSUPPORTED;
    const Layout y = layout(num_seqs);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    ExpandedParams p;
    p.out = static_cast<uint16_t *>(out);
    p.cu_q = cu_q_lens;
    p.cu_k = cu_k_lens;
    p.seqs = reinterpret_cast<int4 *>(ws);
    p.before = reinterpret_cast<int32_t *>(ws + y.before);
    p.next = reinterpret_cast<int32_t *>(ws + y.next);
    p.num_seqs = num_seqs;
    p.rows = total_q_tokens;
    p.keys = total_k_tokens;
    p.heads = num_heads;
    p.scale_log2 = scale * LOG2E;
    CUtensorMap qmap, kvmap, rmap;
    // (without any key nothing of kv is needed, but a map wants an extent: the
    // query tensor stands in, its values masked)
    const bool none = total_k_tokens == 0;
    if (!pkv_host::encode_tmap_2d(&qmap, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)num_heads * QKD, total_q_tokens,
                                  (uint64_t)num_heads * QKD * 2, 64, BM, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !pkv_host::encode_tmap_2d(&kvmap, none ? q : kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                  none ? (uint64_t)num_heads * QKD : (uint64_t)num_heads * 2 * D, none ? 1 : total_k_tokens,
                                  (uint64_t)num_heads * (none ? QKD : 2 * D) * 2, 64, BN, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !pkv_host::encode_tmap_2d(&rmap, none ? q : k_rope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ROPE,
                                  none ? 1 : total_k_tokens, (uint64_t)(none ? QKD : k_rope_stride) * 2, 64, BN,
                                  CU_TENSOR_MAP_SWIZZLE_128B))
        return KV_ERR_CUDA;
    if (pkv_host::ensure_dynamic_smem<expanded_kernel>(SMEM_BYTES) != cudaSuccess) return KV_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int grid = (int)std::min<int64_t>(items, 152);
    p.grid = grid;
    p.max_items = (int)items;
    p.small = num_seqs <= 32 && items <= 4 * 152;
    if ((!p.small && pkv_host::launch_ex(expanded_plan_kernel, dim3(1), dim3(1024), 0, st, true, p) != cudaSuccess) ||
        pkv_host::launch_ex(expanded_kernel, dim3(grid), dim3(THREADS), SMEM_BYTES, st, true, qmap, kvmap, rmap, p) != cudaSuccess)
        return KV_ERR_CUDA;
    return KV_OK;
}

}  // extern "C"
