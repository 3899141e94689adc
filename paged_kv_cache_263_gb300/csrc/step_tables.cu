// step_tables.cu -- block tables and slot numbers of one serving step, built on
// the device from request lengths (sm_103a).
//
// Sequence s holds c_s tokens and gains n_s.  Its blocks cover ceil(c_s / 16)
// tokens now and ceil((c_s + n_s) / 16) after the step; the difference is taken
// from the caller's list of free blocks, in sequence order:
//   need_s = ceil((c_s + n_s) / 16) - ceil(c_s / 16),  off_s = sum_{r < s} need_r
//   table[s][ceil(c_s / 16) + j] = free[off_s + j],    cu_s = sum_{r < s} n_r
// and row cu_s + i of the step is token c_s + i, in slot
// table[s][(c_s + i) / 16] * 16 + (c_s + i) % 16.
//
// The whole step moves 16 bytes a sequence, 8 a new block and 12 a token: it is
// bound by latency, not bandwidth (64 sequences: 2 KB).  So it is one launch:
// every CTA computes both prefix sums over all sequences by itself (they are
// read from L2, CHUNK sequences at a time), keeps them in shared memory, and then
// writes a share of the rows and of the new blocks, finding each one's sequence
// by a binary search there.  A second launch that consumed the sums would cost
// more than the CTAs' repeated reads (4,096 sequences: 32 KB a CTA).
// 64 sequences with a token each: 5.6 us; 4,096 with up to 33: 12.3 us.
#include "common.cuh"
#include "trace.h"

#include <algorithm>

namespace {

__device__ uint32_t g_status;

using namespace pkv;

constexpr int THREADS = 1024, PER = 2, CHUNK = THREADS * PER;   // sequences in shared memory at a time
constexpr int ROWS_PER_CTA = 1024;

struct StepParams {
    int32_t *tables;
    const int32_t *ctx, *news, *free_ids;
    int32_t *cu, *lens, *positions, *totals;
    int64_t *slots;
    int num_seqs, max_blocks, num_free, num_blocks, max_tokens;
};

__device__ __forceinline__ void flag(uint32_t bits) { atomicOr(&g_status, bits); }

// exclusive prefix sums of a and b over the block (one value a thread), added to
// by the running totals; returns the block's sums
struct Pair {
    long long a, b;
};
__device__ __forceinline__ Pair block_scan(Pair &v, Pair *warp_sums)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    Pair x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ta = __shfl_up_sync(0xffffffffu, x.a, o), tb = __shfl_up_sync(0xffffffffu, x.b, o);
        if (lane >= o) {
            x.a += ta;
            x.b += tb;
        }
    }
    __syncthreads();                       // the sums of the scan before have been read
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    Pair t = warp_sums[lane];              // 32 warps: one sum a lane
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ta = __shfl_up_sync(0xffffffffu, t.a, o), tb = __shfl_up_sync(0xffffffffu, t.b, o);
        if (lane >= o) {
            t.a += ta;
            t.b += tb;
        }
    }
    const Pair all = {__shfl_sync(0xffffffffu, t.a, 31), __shfl_sync(0xffffffffu, t.b, 31)};
    const long long ba = __shfl_sync(0xffffffffu, t.a, (w + 31) & 31), bb = __shfl_sync(0xffffffffu, t.b, (w + 31) & 31);
    v.a = x.a - v.a + (w ? ba : 0);
    v.b = x.b - v.b + (w ? bb : 0);
    return all;
}

// the last i in [0, n) with v[i] <= x (v non-decreasing, v[0] <= x)
__device__ __forceinline__ int last_at_most(const int *v, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(THREADS) step_tables_kernel(const StepParams p)
{
    __shared__ Pair warp_sums[32];
    __shared__ int sh_cu[CHUNK + 1], sh_off[CHUNK + 1];
    __shared__ int sh_ctx[CHUNK];          // tokens held, or -1: the sequence was refused
    __shared__ int sh_taken;
    griddep_launch_dependents();
    const int tid = threadIdx.x, G = gridDim.x;
    const bool first = blockIdx.x == 0;
    const long long gid = (long long)blockIdx.x * THREADS + tid, gstep = (long long)G * THREADS;
    if (tid == 0) sh_taken = 0;
    long long rows_all = 0, need_all = 0;  // of every valid sequence before the chunk, refused ones among them
    long long rows = 0;                    // of the accepted ones
    uint32_t bad = 0;
    for (int base = 0; base < p.num_seqs; base += CHUNK) {
        const int cnt = min(CHUNK, p.num_seqs - base);
        int c[PER], n[PER], need[PER];
        Pair mine = {0, 0};
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = tid * PER + k;
            c[k] = n[k] = need[k] = 0;
            if (i < cnt) {
                c[k] = p.ctx[base + i];
                n[k] = p.news[base + i];
                // (64 bits: the sum of two lengths may pass 32)
                if (c[k] < 0 || n[k] < 0 || (long long)c[k] + n[k] > (long long)p.max_blocks * BS) {
                    bad |= ST_BAD_LEN;
                    n[k] = -1;
                } else {
                    need[k] = (int)(((long long)c[k] + n[k] + BS - 1) / BS - ((long long)c[k] + BS - 1) / BS);
                    mine.a += n[k];
                    mine.b += need[k];
                }
            }
        }
        Pair at = mine;
        const Pair all = block_scan(at, warp_sums);
        // refused: the rows (blocks) of it and of every valid sequence before it
        // are more than max_tokens (the free list) holds
        Pair run = {at.a + rows_all, at.b + need_all};
        bool ok[PER];
        int taken = 0;
        Pair acc = {0, 0};
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = tid * PER + k;
            ok[k] = false;
            if (i < cnt) {
                const int rn = max(n[k], 0);
                ok[k] = n[k] >= 0;
                if (rn > 0 && run.a + rn > p.max_tokens) {
                    ok[k] = false;
                    bad |= ST_BAD_LEN;
                }
                if (need[k] > 0 && run.b + need[k] > p.num_free) {
                    ok[k] = false;
                    bad |= ST_NO_BLOCKS;
                }
                sh_off[i] = (int)min(run.b, (long long)INT_MAX);
                sh_ctx[i] = ok[k] ? c[k] : -1;
                run.a += rn;
                run.b += need[k];
                if (ok[k]) {
                    acc.a += rn;
                    if (need[k] > 0) taken = (int)run.b;
                }
            }
        }
        if (taken > 0) atomicMax(&sh_taken, taken);
        // the accepted sequences' rows: the first sums, unless one was refused
        Pair at2 = acc, all2 = all;
        if (__syncthreads_or(mine.a != acc.a)) all2 = block_scan(at2, warp_sums);
        else at2.a = at.a;
        long long r = rows + at2.a;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = tid * PER + k;
            if (i < cnt) {
                sh_cu[i] = (int)r;
                if (first) {
                    p.cu[base + i] = (int)r;
                    p.lens[base + i] = c[k] + (ok[k] ? n[k] : 0);
                }
                if (ok[k]) r += n[k];
            }
        }
        const long long rows_end = rows + all2.a, need_end = need_all + all.b;
        __syncthreads();
        // the new blocks of this chunk, by their place in the free list
        const long long blk_end = min(need_end, (long long)p.num_free);
        for (long long x = need_all + gid; x < blk_end; x += gstep) {
            const int i = last_at_most(sh_off, cnt, (int)x);
            if (sh_ctx[i] < 0) continue;
            const int have = (int)(((long long)sh_ctx[i] + BS - 1) / BS);
            p.tables[(size_t)(base + i) * p.max_blocks + have + ((int)x - sh_off[i])] = p.free_ids[x];
        }
        // its rows
        for (long long t = rows + gid; t < rows_end; t += gstep) {
            const int i = last_at_most(sh_cu, cnt, (int)t);
            const int ctx = sh_ctx[i], pos = ctx + ((int)t - sh_cu[i]), blk = pos / BS;
            const int have = (int)(((long long)ctx + BS - 1) / BS);
            const int id = blk < have ? p.tables[(size_t)(base + i) * p.max_blocks + blk]
                                      : p.free_ids[sh_off[i] + (blk - have)];
            const bool in_pool = id >= 0 && id < p.num_blocks;
            if (!in_pool) flag(ST_BAD_BLOCK);
            p.slots[t] = in_pool ? (int64_t)id * BS + pos % BS : -1;
            p.positions[t] = pos;
        }
        rows = rows_end;
        rows_all += all.a;
        need_all = need_end;
        __syncthreads();                   // the shared tables are rewritten by the next chunk
    }
    // rows past the step's last: no slot, position 0
    for (long long t = rows + gid; t < p.max_tokens; t += gstep) {
        p.slots[t] = -1;
        p.positions[t] = 0;
    }
    if (first) {
        if (bad) flag(bad);
        if (tid == 0) {
            p.cu[p.num_seqs] = (int)rows;
            p.totals[0] = (int)rows;
            p.totals[1] = sh_taken;
        }
    }
}

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return x < y + nb && y < x + na;
}

}  // namespace

namespace pkv_step {
cudaError_t status_word(uint32_t **at) { return cudaGetSymbolAddress(reinterpret_cast<void **>(at), g_status); }
}  // namespace pkv_step

extern "C" kv_status kv_build_step_tables(int32_t *block_tables, int32_t max_blocks_per_seq,
                                          const int32_t *context_lens, const int32_t *new_lens, int32_t num_seqs,
                                          const int32_t *free_blocks, int32_t num_free, int32_t num_blocks,
                                          int32_t *cu_q_lens, int32_t *total_lens, int64_t *slot_mapping,
                                          int32_t *positions, int32_t max_tokens, int32_t *totals, void *stream)
{
    PKV_NVTX_RANGE("kv_build_step_tables");
    if (num_seqs < 0 || max_blocks_per_seq < 1 || max_blocks_per_seq > INT32_MAX / BS || num_free < 0 ||
        num_blocks < 1 || num_blocks > INT32_MAX / BS || max_tokens < 0)
        return KV_ERR_INVALID;
    if (!cu_q_lens || !totals) return KV_ERR_INVALID;
    if (num_seqs > 0 && (!block_tables || !context_lens || !new_lens || !total_lens)) return KV_ERR_INVALID;
    if ((num_free > 0 && !free_blocks) || (max_tokens > 0 && (!slot_mapping || !positions))) return KV_ERR_INVALID;
    // (the CTAs read the inputs at different times, so no output may lie over one, or over another output)
    const struct { const void *p; size_t n, align; bool out; } b[] = {
        {context_lens, 4ull * num_seqs, 4, false}, {new_lens, 4ull * num_seqs, 4, false},
        {free_blocks, 4ull * num_free, 4, false},
        {block_tables, 4ull * num_seqs * max_blocks_per_seq, 4, true}, {cu_q_lens, 4ull * num_seqs + 4, 4, true},
        {total_lens, 4ull * num_seqs, 4, true}, {slot_mapping, 8ull * max_tokens, 8, true},
        {positions, 4ull * max_tokens, 4, true}, {totals, 8, 4, true}};
    for (const auto &x : b) {
        if (x.n && !pkv_host::aligned(x.p, x.align)) return KV_ERR_INVALID;
        for (const auto &y : b)
            if (&x != &y && x.out && x.n && y.n && overlap(x.p, x.n, y.p, y.n)) return KV_ERR_INVALID;
    }
    StepParams p = {block_tables, context_lens, new_lens, free_blocks, cu_q_lens, total_lens, positions, totals,
                    slot_mapping, num_seqs, max_blocks_per_seq, num_free, num_blocks, max_tokens};
    // a CTA for every ROWS_PER_CTA rows (or new blocks: at most one a row and one a sequence), at most one an SM
    const long long want = ((long long)std::max(max_tokens, std::min(num_free, num_seqs)) + ROWS_PER_CTA - 1) / ROWS_PER_CTA;
    const int grid = (int)std::max(1ll, std::min(want, 152ll));
    step_tables_kernel<<<grid, THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}
