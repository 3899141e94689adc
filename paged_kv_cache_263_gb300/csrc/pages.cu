// pages.cu -- operations on whole blocks of paged caches and on the tables that
// reach them (sm_103a): copies of many blocks over many caches, forks of
// sequences, and the rewriting of tables after blocks have moved.
//
// Samples of one prompt share its blocks, and a writer into a shared block first
// gets its own copy ("Waste, and three ways to reclaim it", section "Sharing, and
// what makes a prefix reusable"; "M.65 Inference serving", block management (e),
// (g)).  kv_copy_on_write does this for one block and one layer; a fork of a whole
// batch needs one block a sequence copied in every layer, with the sequences'
// ancestors known on the device only (beam search chooses them there).
#include "common.cuh"
#include "trace.h"

#include <algorithm>

namespace {

__device__ uint32_t g_status;

using namespace pkv;

__device__ __forceinline__ void flag(uint32_t bits) { atomicOr(&g_status, bits); }

// These kernels are short, and their launches follow one another (a fork, its copies,
// the attention): each is launched programmatically, and waits here before its first
// access to memory.  (Plain loads behind it: what a kernel before wrote is not constant
// for as long as this one is resident.)
__device__ __forceinline__ void begin()
{
    griddep_launch_dependents();
    griddep_wait();
}

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return x < y + nb && y < x + na;
}

// -------------------------------------------------------------- block copies
constexpr int COPY_THREADS = 256, COPY_UNROLL = 4, COPY_CACHES = 128;
struct CopyParams {
    uint4 *cache[COPY_CACHES];
    const int32_t *src, *dst;
    int64_t units;         // 16-byte units of a block
    int num_blocks, pieces;
};

// A CTA copies one piece, at most 16 KiB, of one block of one cache (grid: pieces of
// the pairs, caches): every thread has all its loads in flight before its first store,
// and CTAs that come and go keep the loads of some beside the stores of others.  Bound
// by memory.  512 blocks of 32 KiB in 32 caches: 155 us, 6.9 TB/s read and written,
// where a grid of 8 CTAs an SM that loop over the pieces took 176 us, and this one
// with the caches varying fastest 162 us.
__global__ void __launch_bounds__(COPY_THREADS) copy_blocks_kernel(const __grid_constant__ CopyParams p)
{
    begin();
    const int i = blockIdx.x / p.pieces, piece = blockIdx.x - i * p.pieces;
    const int s = p.src[i], d = p.dst[i];
    if (d < 0 && s < 0) return;          // no pair
    if (s < 0 || d < 0 || s >= p.num_blocks || d >= p.num_blocks) {
        if (threadIdx.x == 0) flag(ST_BAD_BLOCK);
        return;
    }
    if (s == d) return;
    const int64_t each = (p.units + p.pieces - 1) / p.pieces;   // at most COPY_THREADS x COPY_UNROLL
    const uint4 *from = p.cache[blockIdx.y] + s * p.units;
    uint4 *to = p.cache[blockIdx.y] + d * p.units;
    const int64_t u0 = piece * each + threadIdx.x, u1 = min(p.units, (piece + 1) * each);
    uint4 v[COPY_UNROLL];
#pragma unroll
    for (int r = 0; r < COPY_UNROLL; ++r)
        if (u0 + r * COPY_THREADS < u1) v[r] = from[u0 + r * COPY_THREADS];
#pragma unroll
    for (int r = 0; r < COPY_UNROLL; ++r)
        if (u0 + r * COPY_THREADS < u1) to[u0 + r * COPY_THREADS] = v[r];
}

// -------------------------------------------------------------------- forks
constexpr int FORK_THREADS = 1024, FORK_MAX = 16384;   // parents and children at most
struct ForkParams {
    const int32_t *tables, *lens, *parents, *free_ids;
    int32_t *child_tables, *child_lens, *src, *dst, *taken;
    int max_blocks, num_parents, num_children, num_free, first_keeps;
};
// a parent's first child (32 bits), a child's length (32), parent and fresh block (16 each)
constexpr int fork_smem(int parents, int children) { return 4 * parents + 8 * children; }

// Every CTA finds, for all children, which of them take a fresh block and the
// place of it in the free list (a scan), then writes a share of the rows, a warp a
// row.  What it reads of the batch it reads once, into shared memory; the whole call
// moves little and is bound by the chain of its memory trips (parents, lengths, rows).
__global__ void __launch_bounds__(FORK_THREADS) fork_tables_kernel(const ForkParams p)
{
    extern __shared__ int32_t sh[];
    __shared__ int32_t warp_sums[FORK_THREADS / 32];
    int32_t *first = sh, *len = sh + p.num_parents;
    int16_t *parent = reinterpret_cast<int16_t *>(len + p.num_children), *place = parent + p.num_children;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    begin();
    // lengths and parents of all children; -1: the child is refused
    for (int c = tid; c < p.num_children; c += FORK_THREADS) {
        const int a = p.parents[c];
        int L = -1;
        if (a >= 0 && a < p.num_parents) L = p.lens[a];
        if (L < 0 || L > p.max_blocks * BS) L = -1;
        parent[c] = (int16_t)(L < 0 ? 0 : a);
        len[c] = L;
    }
    if (p.first_keeps) {
        for (int i = tid; i < p.num_parents; i += FORK_THREADS) first[i] = INT_MAX;
        __syncthreads();
        for (int c = tid; c < p.num_children; c += FORK_THREADS)
            if (len[c] >= 0) atomicMin(&first[parent[c]], c);
    }
    __syncthreads();
    int taken = 0;
    for (int base = 0; base < p.num_children; base += FORK_THREADS) {
        const int c = base + tid;
        const bool fresh = c < p.num_children && len[c] > 0 && len[c] % BS && !(p.first_keeps && first[parent[c]] == c);
        const unsigned m = __ballot_sync(0xffffffffu, fresh);
        if (lane == 0) warp_sums[w] = __popc(m);
        __syncthreads();
        // (32 warps: one sum a lane)
        int v = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
        }
        const int before = w ? __shfl_sync(0xffffffffu, v, (w + 31) & 31) : 0;
        if (c < p.num_children) place[c] = (int16_t)(fresh ? taken + before + __popc(m & ((1u << lane) - 1u)) : -1);
        taken += __shfl_sync(0xffffffffu, v, 31);
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) *p.taken = min(taken, p.num_free);
    const int warps = FORK_THREADS / 32;
    for (int c = blockIdx.x * warps + w; c < p.num_children; c += gridDim.x * warps) {
        const int L = len[c], at = place[c];
        const bool ok = L >= 0 && at < p.num_free;
        if (!ok && lane == 0) flag(L < 0 ? ST_BAD_LEN : ST_NO_BLOCKS);
        const int n = ok ? (L + BS - 1) / BS : 0, kept = at >= 0 ? n - 1 : n;
        const int32_t *from = p.tables + (size_t)parent[c] * p.max_blocks;
        int32_t *to = p.child_tables + (size_t)c * p.max_blocks;
        int s = -1, d = -1;
        if (lane == 0 && ok && at >= 0) {
            s = from[n - 1];
            d = p.free_ids[at];
        }
        // (eight entries a lane in flight)
        for (int j0 = lane; j0 < kept; j0 += 256) {
            int32_t e[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j0 + 32 * u < kept) e[u] = from[j0 + 32 * u];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j0 + 32 * u < kept) to[j0 + 32 * u] = e[u];
        }
        if (lane == 0) {
            if (ok && at >= 0) to[n - 1] = d;
            p.src[c] = s;
            p.dst[c] = d;
            p.child_lens[c] = ok ? L : 0;
        }
    }
}

// ------------------------------------------------------------- table rewriting
// A CTA takes REMAP_PIECE entries of a row at a time.  Entries outside the range of
// the moved ids are done with two comparisons -- a compaction moves the pool's upper
// end, so nearly all of them -- and the others look their id up in the list.  Bound by
// latency: 512 rows of up to 2,048 entries take 2.2 us with no entry in the range, and 8.7
// with 8,192 that are moved, by the 13 steps of each search, a memory trip each, one after
// another for the entries of a warp (16 rows, 9 moves: 1.4 and 1.8).
constexpr int REMAP_THREADS = 256, REMAP_UNROLL = 4, REMAP_PIECE = REMAP_THREADS * REMAP_UNROLL;
__global__ void __launch_bounds__(REMAP_THREADS)
    remap_tables_kernel(int32_t *tables, int max_blocks, const int32_t *lens, int num_seqs, const int32_t *src,
                        const int32_t *dst, int n, int pieces)
{
    begin();
    const int lowest = *src, highest = src[n - 1];
    for (int64_t x = blockIdx.x; x < (int64_t)num_seqs * pieces; x += gridDim.x) {
        const int s = (int)(x / pieces), piece = (int)(x - (int64_t)s * pieces);
        int32_t *row = tables + (size_t)s * max_blocks;
        const int L = lens[s], j0 = piece * REMAP_PIECE + threadIdx.x;
        int32_t id[REMAP_UNROLL];
        // (asked for together with the length: entries past it are not used)
#pragma unroll
        for (int u = 0; u < REMAP_UNROLL; ++u)
            if (j0 + u * REMAP_THREADS < max_blocks) id[u] = row[j0 + u * REMAP_THREADS];
        if (L < 0 || L > max_blocks * BS) {
            if (piece == 0 && threadIdx.x == 0) flag(ST_BAD_LEN);
            continue;
        }
        const int used = (L + BS - 1) / BS;
#pragma unroll
        for (int u = 0; u < REMAP_UNROLL; ++u) {
            const int j = j0 + u * REMAP_THREADS;
            if (j >= used || id[u] < lowest || id[u] > highest) continue;
            int lo = 0, hi = n;
            while (hi - lo > 1) {
                const int mid = lo + ((hi - lo) >> 1);
                if (src[mid] <= id[u]) lo = mid;
                else hi = mid;
            }
            if (src[lo] == id[u]) row[j] = dst[lo];
        }
    }
}

}  // namespace

namespace pkv_pages {
cudaError_t status_word(uint32_t **at) { return cudaGetSymbolAddress(reinterpret_cast<void **>(at), g_status); }
}  // namespace pkv_pages

extern "C" {

kv_status kv_copy_blocks(void *const *caches, int32_t num_caches, int64_t block_bytes, int32_t num_blocks,
                         const int32_t *src, const int32_t *dst, int32_t n, void *stream)
{
    PKV_NVTX_RANGE("kv_copy_blocks");
    if (num_caches < 0 || n < 0 || num_blocks < 1 || block_bytes < 16 || block_bytes % 16) return KV_ERR_INVALID;
    if (num_caches == 0 || n == 0) return KV_OK;
    if (!caches || !src || !dst || !pkv_host::aligned(src, 4) || !pkv_host::aligned(dst, 4)) return KV_ERR_INVALID;
    if (block_bytes > INT64_MAX / num_blocks) return KV_ERR_INVALID;
    for (int i = 0; i < num_caches; ++i)
        if (!caches[i] || !pkv_host::aligned(caches[i], 16)) return KV_ERR_INVALID;
    CopyParams p;
    p.src = src;
    p.dst = dst;
    p.units = block_bytes / 16;
    p.num_blocks = num_blocks;
    const int64_t pieces = (p.units + COPY_THREADS * COPY_UNROLL - 1) / (COPY_THREADS * COPY_UNROLL);
    if (pieces > INT32_MAX / n) return KV_ERR_UNSUPPORTED;
    p.pieces = (int)pieces;
    for (int at = 0; at < num_caches; at += COPY_CACHES) {
        const int count = std::min(num_caches - at, COPY_CACHES);
        for (int i = 0; i < count; ++i) p.cache[i] = static_cast<uint4 *>(caches[at + i]);
        if (pkv_host::launch_ex(copy_blocks_kernel, dim3((unsigned)(n * pieces), (unsigned)count), dim3(COPY_THREADS), 0,
                                static_cast<cudaStream_t>(stream), true, p) != cudaSuccess)
            return KV_ERR_CUDA;
    }
    return KV_OK;
}

kv_status kv_fork_tables(const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens,
                         int32_t num_parents, const int32_t *parents, int32_t num_children, int32_t first_keeps,
                         const int32_t *free_blocks, int32_t num_free, int32_t *child_tables, int32_t *child_lens,
                         int32_t *copy_src, int32_t *copy_dst, int32_t *taken, void *stream)
{
    PKV_NVTX_RANGE("kv_fork_tables");
    if (num_parents < 0 || num_children < 0 || num_free < 0 || max_blocks_per_seq < 1 ||
        max_blocks_per_seq > INT32_MAX / BS)
        return KV_ERR_INVALID;
    if (num_parents > FORK_MAX || num_children > FORK_MAX) return KV_ERR_UNSUPPORTED;
    if (!taken || (num_parents > 0 && (!block_tables || !context_lens)) || (num_free > 0 && !free_blocks) ||
        (num_children > 0 && (!parents || !child_tables || !child_lens || !copy_src || !copy_dst)))
        return KV_ERR_INVALID;
    const size_t np = num_parents, nc = num_children;
    const struct { const void *p; size_t n; bool out; } b[] = {
        {block_tables, 4 * np * max_blocks_per_seq, false}, {context_lens, 4 * np, false}, {parents, 4 * nc, false},
        {free_blocks, 4ull * num_free, false}, {child_tables, 4 * nc * max_blocks_per_seq, true},
        {child_lens, 4 * nc, true}, {copy_src, 4 * nc, true}, {copy_dst, 4 * nc, true}, {taken, 4, true}};
    for (const auto &x : b) {
        if (x.n && !pkv_host::aligned(x.p, 4)) return KV_ERR_INVALID;
        for (const auto &y : b)
            if (&x != &y && x.out && x.n && y.n && overlap(x.p, x.n, y.p, y.n)) return KV_ERR_INVALID;
    }
    const ForkParams p = {block_tables, context_lens, parents, free_blocks, child_tables, child_lens, copy_src, copy_dst,
                          taken, max_blocks_per_seq, num_parents, num_children, num_free, first_keeps != 0};
    const int smem = fork_smem(num_parents, num_children);
    if (pkv_host::ensure_dynamic_smem<fork_tables_kernel>(fork_smem(FORK_MAX, FORK_MAX)) != cudaSuccess) return KV_ERR_CUDA;
    const int warps = FORK_THREADS / 32;
    const int grid = std::max(1, std::min((num_children + warps - 1) / warps, 152));
    return pkv_host::launch_ex(fork_tables_kernel, dim3(grid), dim3(FORK_THREADS), smem, static_cast<cudaStream_t>(stream),
                               true, p) == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

kv_status kv_remap_tables(int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens,
                          int32_t num_seqs, const int32_t *src, const int32_t *dst, int32_t n, void *stream)
{
    PKV_NVTX_RANGE("kv_remap_tables");
    if (num_seqs < 0 || n < 0 || max_blocks_per_seq < 1 || max_blocks_per_seq > INT32_MAX / BS) return KV_ERR_INVALID;
    if (num_seqs == 0 || n == 0) return KV_OK;
    if (!block_tables || !context_lens || !src || !dst) return KV_ERR_INVALID;
    const size_t t = 4ull * num_seqs * max_blocks_per_seq;
    const struct { const void *p; size_t n; } in[] = {{context_lens, 4ull * num_seqs}, {src, 4ull * n}, {dst, 4ull * n}};
    if (!pkv_host::aligned(block_tables, 4)) return KV_ERR_INVALID;
    for (const auto &x : in)
        if (!pkv_host::aligned(x.p, 4) || overlap(block_tables, t, x.p, x.n)) return KV_ERR_INVALID;
    const int pieces = (max_blocks_per_seq + REMAP_PIECE - 1) / REMAP_PIECE;
    const int grid = (int)std::min<int64_t>((int64_t)num_seqs * pieces, 152 * 8);
    return pkv_host::launch_ex(remap_tables_kernel, dim3(grid), dim3(REMAP_THREADS), 0, static_cast<cudaStream_t>(stream),
                               true, block_tables, max_blocks_per_seq, context_lens, num_seqs, src, dst, n, pieces) ==
                   cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

}  // extern "C"
