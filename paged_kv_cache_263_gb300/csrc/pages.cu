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
    int n, num_caches, num_blocks, pieces;
};

// A CTA copies a piece of at most 16 KiB of one block of one cache at a time: every
// thread has COPY_UNROLL loads in flight before its first store.
__global__ void __launch_bounds__(COPY_THREADS) copy_blocks_kernel(const __grid_constant__ CopyParams p)
{
    const int64_t total = (int64_t)p.n * p.num_caches * p.pieces;
    const int64_t each = (p.units + p.pieces - 1) / p.pieces;
    for (int64_t x = blockIdx.x; x < total; x += gridDim.x) {
        const int64_t y = x / p.pieces;
        const int piece = (int)(x - y * p.pieces), c = (int)(y % p.num_caches), i = (int)(y / p.num_caches);
        const int s = __ldg(p.src + i), d = __ldg(p.dst + i);
        if (d < 0 && s < 0) continue;          // no pair
        if (s < 0 || d < 0 || s >= p.num_blocks || d >= p.num_blocks) {
            if (threadIdx.x == 0) flag(ST_BAD_BLOCK);
            continue;
        }
        if (s == d) continue;
        const uint4 *from = p.cache[c] + s * p.units;
        uint4 *to = p.cache[c] + d * p.units;
        const int64_t u0 = piece * each + threadIdx.x, u1 = min(p.units, (piece + 1) * each);
        uint4 v[COPY_UNROLL];
#pragma unroll
        for (int r = 0; r < COPY_UNROLL; ++r)
            if (u0 + r * COPY_THREADS < u1) v[r] = from[u0 + r * COPY_THREADS];
#pragma unroll
        for (int r = 0; r < COPY_UNROLL; ++r)
            if (u0 + r * COPY_THREADS < u1) to[u0 + r * COPY_THREADS] = v[r];
    }
}

// -------------------------------------------------------------------- forks
constexpr int FORK_THREADS = 512, FORK_MAX = 16384;   // parents and children at most
struct ForkParams {
    const int32_t *tables, *lens, *parents, *free_ids;
    int32_t *child_tables, *child_lens, *src, *dst, *taken;
    int max_blocks, num_parents, num_children, num_free, first_keeps;
};

// Every CTA finds, for all children, which of them take a fresh block and the
// place of it in the free list (a scan), then writes a share of the rows, a warp a
// row.
__global__ void __launch_bounds__(FORK_THREADS) fork_tables_kernel(const ForkParams p)
{
    extern __shared__ int32_t sh[];
    __shared__ int32_t warp_sums[FORK_THREADS / 32];
    int32_t *first = sh, *place = sh + p.num_parents;   // a parent's first child; a child's fresh block, or -1
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    for (int i = tid; i < p.num_parents; i += FORK_THREADS) first[i] = INT_MAX;
    __syncthreads();
    if (p.first_keeps) {
        for (int c = tid; c < p.num_children; c += FORK_THREADS) {
            const int a = p.parents[c];
            if (a >= 0 && a < p.num_parents) atomicMin(&first[a], c);
        }
        __syncthreads();
    }
    int taken = 0;
    for (int base = 0; base < p.num_children; base += FORK_THREADS) {
        const int c = base + tid;
        bool fresh = false;
        if (c < p.num_children) {
            const int a = p.parents[c];
            if (a >= 0 && a < p.num_parents) {
                const int L = p.lens[a];
                fresh = L > 0 && L <= p.max_blocks * BS && L % BS && first[a] != c;
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, fresh);
        if (lane == 0) warp_sums[w] = __popc(m);
        __syncthreads();
        int before = taken, all = 0;
        for (int i = 0; i < FORK_THREADS / 32; ++i) {
            if (i == w) before += all;
            all += warp_sums[i];
        }
        if (c < p.num_children) place[c] = fresh ? before + __popc(m & ((1u << lane) - 1u)) : -1;
        taken += all;
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) *p.taken = min(taken, p.num_free);
    const int warps = FORK_THREADS / 32;
    for (int c = blockIdx.x * warps + w; c < p.num_children; c += gridDim.x * warps) {
        const int a = p.parents[c];
        int L = -1;
        if (a >= 0 && a < p.num_parents) L = p.lens[a];
        bool ok = L >= 0 && L <= p.max_blocks * BS;
        if (!ok && lane == 0) flag(ST_BAD_LEN);
        const int at = place[c];
        if (ok && at >= p.num_free) {
            ok = false;
            if (lane == 0) flag(ST_NO_BLOCKS);
        }
        const int n = ok ? (L + BS - 1) / BS : 0;
        const int32_t *from = p.tables + (size_t)max(a, 0) * p.max_blocks;
        int32_t *to = p.child_tables + (size_t)c * p.max_blocks;
        const int kept = ok && at >= 0 ? n - 1 : n;
        for (int j = lane; j < kept; j += 32) to[j] = from[j];
        if (lane == 0) {
            int s = -1, d = -1;
            if (kept < n) {
                s = from[n - 1];
                d = p.free_ids[at];
                to[n - 1] = d;
            }
            p.src[c] = s;
            p.dst[c] = d;
            p.child_lens[c] = ok ? L : 0;
        }
    }
}

// ------------------------------------------------------------- table rewriting
constexpr int REMAP_THREADS = 256;
__global__ void __launch_bounds__(REMAP_THREADS)
    remap_tables_kernel(int32_t *__restrict__ tables, int max_blocks, const int32_t *__restrict__ lens, int num_seqs,
                        const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int n)
{
    for (int s = blockIdx.x; s < num_seqs; s += gridDim.x) {
        const int L = lens[s];
        if (L < 0 || L > max_blocks * BS) {
            if (threadIdx.x == 0) flag(ST_BAD_LEN);
            continue;
        }
        const int used = (L + BS - 1) / BS;
        for (int j = threadIdx.x; j < used; j += REMAP_THREADS) {
            int32_t *e = tables + (size_t)s * max_blocks + j;
            const int id = *e;
            int lo = 0, hi = n;
            while (hi - lo > 1) {
                const int mid = lo + ((hi - lo) >> 1);
                if (__ldg(src + mid) <= id) lo = mid;
                else hi = mid;
            }
            if (__ldg(src + lo) == id) *e = __ldg(dst + lo);
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
    p.n = n;
    p.num_blocks = num_blocks;
    const int64_t pieces = (p.units + COPY_THREADS * COPY_UNROLL - 1) / (COPY_THREADS * COPY_UNROLL);
    if (pieces > INT32_MAX) return KV_ERR_UNSUPPORTED;
    p.pieces = (int)pieces;
    for (int at = 0; at < num_caches; at += COPY_CACHES) {
        p.num_caches = std::min(num_caches - at, COPY_CACHES);
        for (int i = 0; i < p.num_caches; ++i) p.cache[i] = static_cast<uint4 *>(caches[at + i]);
        const int64_t want = std::min<int64_t>((int64_t)n * p.num_caches, 152 * 8) * std::min<int64_t>(pieces, 152 * 8);
        const int grid = (int)std::min<int64_t>(want, 152 * 8);
        copy_blocks_kernel<<<grid, COPY_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
        if (cudaGetLastError() != cudaSuccess) return KV_ERR_CUDA;
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
    const int smem = (num_parents + num_children) * 4;
    if (pkv_host::ensure_dynamic_smem<fork_tables_kernel>(2 * FORK_MAX * 4) != cudaSuccess) return KV_ERR_CUDA;
    const int warps = FORK_THREADS / 32;
    const int grid = std::max(1, std::min((num_children + warps - 1) / warps, 152));
    fork_tables_kernel<<<grid, FORK_THREADS, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? KV_OK : KV_ERR_CUDA;
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
    remap_tables_kernel<<<std::min(num_seqs, 152 * 8), REMAP_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
        block_tables, max_blocks_per_seq, context_lens, num_seqs, src, dst, n);
    return cudaGetLastError() == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

}  // extern "C"
