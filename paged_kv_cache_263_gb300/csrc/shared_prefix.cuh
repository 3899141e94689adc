// shared_prefix.cuh -- how a batch of sequences in groups with a common prefix is
// described on the device, read alike by the kernel that attends the prefixes, the
// one that attends the tails and the one that joins the two.
//
// Group g holds sequences cu_groups[g] .. cu_groups[g+1]-1 of the batch, and their
// first prefix_lens[g] tokens are the same.  Only whole blocks can be shared, so P =
// prefix_lens[g] rounded down to blocks is attended once, through the table row of
// the group's first sequence; every sequence attends its keys from P on through
// its own row.  Sequences of no group have P = 0.
#pragma once

#include "common.cuh"

#include <cuda_bf16.h>

namespace pkv {

struct SharedBatch {
    const int32_t *cu_groups, *prefix_lens;   // [num_groups + 1], [num_groups]
    const int32_t *cu_q_lens;                 // [num_seqs + 1], or null: one row a sequence
    const int32_t *context_lens;              // [num_seqs]
    int num_groups, num_seqs, total_rows, max_q_len;
    int max_prefix, max_tail;                 // keys, bounds given by the caller (max_prefix in whole blocks)
    int max_blocks;
};

#if defined(__CUDACC__)
// the last i in [0, n) with v[i] <= x, or 0 (bounded whatever v holds; v non-decreasing):
// by the whole warp, a memory round trip for every factor of 32
__device__ __forceinline__ int last_at_most(const int32_t *v, int n, int x, int lane)
{
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) >> 5, i = lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, i < n && v[lo + min(i, n - 1)] <= x);
        const int at = m ? 31 - __clz(m) : 0;
        lo += at * step;
        n = min(step, n - at * step);
    }
    return lo;
}

struct SharedGroup {
    int s0, s1, row0, rows, P;
    bool ok;          // within the batch, the tensors and the caller's bounds
};
__device__ __forceinline__ SharedGroup shared_group(const SharedBatch &b, int g)
{
    SharedGroup r;
    r.s0 = b.cu_groups[g];
    r.s1 = b.cu_groups[g + 1];
    const int p = b.prefix_lens[g];
    r.P = p & ~(BS - 1);
    r.ok = r.s0 >= 0 && r.s0 <= r.s1 && r.s1 <= b.num_seqs && p >= 0 && r.P <= b.max_prefix;
    r.row0 = r.rows = 0;
    if (r.ok && r.s0 < r.s1) {
        const int a = b.cu_q_lens ? b.cu_q_lens[r.s0] : r.s0;
        const int e = b.cu_q_lens ? b.cu_q_lens[r.s1] : r.s1;
        r.ok = a >= 0 && a <= e && e <= b.total_rows;
        r.row0 = a;
        r.rows = r.ok ? e - a : 0;
    }
    return r;
}

enum { SEQ_BAD = 0, SEQ_EMPTY = 1, SEQ_OK = 2 };
struct SharedSeq {
    int state;        // SEQ_BAD: left out; SEQ_EMPTY: no context, its rows are zeros
    int row0, n;      // its query rows
    int L, P;         // context, and how much of it is its group's prefix
    int first;        // the sequence whose table row the prefix is read through
};
// (g: the last group that begins at or before s; any number if there is none)
__device__ __forceinline__ SharedSeq shared_seq_in(const SharedBatch &b, int s, int g)
{
    SharedSeq r;
    r.state = SEQ_BAD;
    // what does not depend on the group is asked for together with it
    r.row0 = b.cu_q_lens ? b.cu_q_lens[s] : s;
    r.n = (b.cu_q_lens ? b.cu_q_lens[s + 1] : s + 1) - r.row0;
    r.L = b.context_lens[s];
    r.P = 0;
    r.first = s;
    bool ok = true;
    if (b.num_groups > 0) {
        const SharedGroup gr = shared_group(b, g);
        if (s >= gr.s0 && s < gr.s1) {
            ok = gr.ok && r.row0 >= gr.row0 && r.row0 + r.n <= gr.row0 + gr.rows;
            r.P = gr.P;
            r.first = gr.s0;
        }
    }
    if (r.row0 < 0 || r.n < 0 || r.row0 > b.total_rows - r.n || r.n > b.max_q_len) return r;
    if (r.L == 0) {
        r.state = SEQ_EMPTY;
        return r;
    }
    // the rows' own tokens lie behind the prefix
    if (!ok || r.L < 0 || r.L > b.max_blocks * BS || r.L - r.n < r.P || r.L - r.P > b.max_tail) return r;
    r.state = SEQ_OK;
    return r;
}
// by the whole warp, for a sequence that is the same in all lanes
__device__ __forceinline__ SharedSeq shared_seq(const SharedBatch &b, int s, int lane)
{
    return shared_seq_in(b, s, b.num_groups > 1 ? last_at_most(b.cu_groups, b.num_groups, s, lane) : 0);
}
// by the whole warp, sequence s0 + lane for each lane (SEQ_BAD past the batch)
__device__ __forceinline__ SharedSeq shared_seq_window(const SharedBatch &b, int s0, int lane)
{
    const int s = s0 + lane;
    int g = 0;
    if (b.num_groups > 1) {
        // the first sequence's group, then the 32 groups' beginnings behind it, counted
        g = last_at_most(b.cu_groups, b.num_groups, s0, lane);
        const int mine = g + 1 + lane < b.num_groups ? b.cu_groups[g + 1 + lane] : INT_MAX;
        int more = 0;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) more += __shfl_sync(0xffffffffu, mine, i) <= s;
        g += more;
        // (empty groups among them: a lane may have further to go, past any number of them)
        for (int end = more == 32 ? b.num_groups : 0; end - g > 1;) {
            const int mid = g + ((end - g) >> 1);
            if (b.cu_groups[mid] <= s) g = mid;
            else end = mid;
        }
    }
    if (s >= b.num_seqs) {
        SharedSeq r = {};
        r.state = SEQ_BAD;
        return r;
    }
    return shared_seq_in(b, s, g);
}
// zeros in the rows of each lane's sequence that is marked (by the whole warp)
__device__ __forceinline__ void zero_rows(__nv_bfloat16 *out, int hq, bool marked, int row0, int n, int lane)
{
    for (unsigned m = __ballot_sync(0xffffffffu, marked); m; m &= m - 1) {
        const int at = __ffs(m) - 1, first = __shfl_sync(0xffffffffu, row0, at), rows = __shfl_sync(0xffffffffu, n, at);
        uint4 *to = reinterpret_cast<uint4 *>(out + (size_t)first * hq * D);
        for (int64_t i = lane; i < (int64_t)rows * hq * (D / 8); i += 32) to[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}
#endif  // __CUDACC__

}  // namespace pkv
