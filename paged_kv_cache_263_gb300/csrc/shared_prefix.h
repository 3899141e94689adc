// shared_prefix.h -- what the host side of attention over shared prefixes
// (shared_prefix.cu) hands to the two kernels that do its products: the chunk
// kernel's shared mode (prefill.cu) for the prefixes, shared_tail.cu for each
// sequence's own keys, or the former for both.
#pragma once

#include "shared_prefix.cuh"

struct SharedCall {
    pkv::SharedBatch b;
    void *out;                        // bf16
    const uint16_t *q;
    const void *k_cache, *v_cache;
    const int32_t *block_tables;
    const float *k_scale, *v_scale;   // fp8 cache
    float *part_o, *part_ml;          // [rows][hq][prefix_splits + tail_splits][128], [..][2] (max, sum)
    int *counter;                     // of the tails' items, set by the kernel before theirs
    int hq, hkv, num_blocks;
    bool fp8, big;                    // big: one query tile a CTA, 128-key tiles
    bool joined;                      // the kernel of the prefixes attends the tails as well
    bool whole;                       // no kernel for the prefixes: the tails' attends whole contexts
    int prefix_splits, prefix_tiles;  // parts of a prefix at most, and KV tiles a part
    int most_parts;                   // parts of a row at most, that the workspace has room for (two or more)
    int64_t prefix_items, tail_items; // work items of prefixes, and of joined tails, at most
    int tail_splits, tail_part_blocks;
    int fine_from, fine_blocks;       // sequences from fine_from on have shorter parts, of fine_blocks
    int sets, set_rows;               // the tails' kernel takes a sequence's rows in sets: how many at most
    double mean_sets;                 // ... and for a sequence of as many rows as there are on average
    float scale_log2;
};

// items of the tails' kernel at most
inline int64_t tail_kernel_items(const SharedCall &c)
{
    const int64_t sets = (int64_t)c.b.num_seqs * c.sets, by_rows = c.b.total_rows / c.set_rows + (int64_t)c.b.num_seqs;
    return (sets < by_rows || c.sets == 1 ? sets : by_rows) * c.hkv * c.tail_splits;
}

// partial results of a row and head; the only one is the output itself
inline int shared_parts(const SharedCall &c) { return c.prefix_splits + c.tail_splits; }

namespace pkv_shared_tail {
// beside: behind the kernel of the prefixes, to run beside it
cudaError_t launch_tails(const SharedCall &c, bool beside, cudaStream_t st);
}  // namespace pkv_shared_tail
namespace pkv_prefill {
// the parts that prefixes are cut into (fields big and prefix_*), and tails where they
// are joined (tail_*)
void plan_prefixes(SharedCall &c, int64_t max_tail);
cudaError_t launch_prefixes(const SharedCall &c, cudaStream_t st);
}  // namespace pkv_prefill
