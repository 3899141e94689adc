// latent_decode.cu -- attention over a paged latent cache, absorbed form
// (sm_103a).
//
// A cached row x_t holds a token's latent (512) and rotary key (64); a head's
// query, multiplied by that head's key expansion beforehand, is 576 wide, and
//   out[r][h] = sum_t p_t x_t[0:512],  p = softmax_t(scale * q[r][h] . x_t)
// over the keys t <= L - n + i that row i of a sequence's n rows sees.
#include "common.cuh"
#include "trace.h"

#include <algorithm>
#include <cmath>

namespace {

__device__ uint32_t g_status;

using namespace pkv;

constexpr float LOG2E = 1.4426950408889634f;

struct LatentParams {
    uint16_t *out;
    const uint16_t *q, *cache;
    const int32_t *cu, *lens, *tables;
    int num_seqs, rows, heads, max_blocks, num_blocks;
    float scale_log2;
};

__device__ __forceinline__ void flag(uint32_t bits) { atomicOr(&g_status, bits); }

// One warp per (row, head): lane l holds dims l, l + 32, ... of q and of the sum.
__global__ void __launch_bounds__(256) latent_simple_kernel(const LatentParams p)
{
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= (long long)p.rows * p.heads) return;
    const int row = (int)(w / p.heads), h = (int)(w % p.heads);
    int s = row, a = row, n = 1;
    if (p.cu) {
        s = -1;
        for (int i = 0; i < p.num_seqs; ++i)
            if (p.cu[i] <= row && row < p.cu[i + 1]) {
                s = i;
                a = p.cu[i];
                n = p.cu[i + 1] - a;
                break;
            }
        if (s < 0) return;
    }
    const int L = p.lens[s];
    if (L < 0 || L > p.max_blocks * BS || (L < n && L != 0) || a < 0 || a + n > p.rows) {
        if (lane == 0) flag(ST_BAD_LEN);
        return;
    }
    const int last = L - n + (row - a);
    float q[18], o[16], m = -INFINITY, l = 0.f;
    const uint16_t *qr = p.q + w * LKD;
    for (int k = 0; k < 18; ++k) q[k] = __uint_as_float((uint32_t)qr[lane + 32 * k] << 16);
    for (int k = 0; k < 16; ++k) o[k] = 0.f;
    for (int t = 0; t <= last && L > 0; ++t) {
        const int id = p.tables[(size_t)s * p.max_blocks + t / BS];
        if (id < 0 || id >= p.num_blocks) {
            if (lane == 0) flag(ST_BAD_BLOCK);
            continue;
        }
        const uint16_t *x = p.cache + ((size_t)id * BS + t % BS) * LKD;
        float v[18], d = 0.f;
        for (int k = 0; k < 18; ++k) {
            v[k] = __uint_as_float((uint32_t)x[lane + 32 * k] << 16);
            d += q[k] * v[k];
        }
        for (int b = 16; b > 0; b >>= 1) d += __shfl_xor_sync(0xffffffffu, d, b);
        d *= p.scale_log2;
        const float mn = fmaxf(m, d), c = ex2(m - mn), e = ex2(d - mn);
        l = l * c + e;
        for (int k = 0; k < 16; ++k) o[k] = o[k] * c + e * v[k];
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint16_t *r = p.out + w * LAT;
    for (int k = 0; k < 16; ++k) r[lane + 32 * k] = (uint16_t)(pack_bf16(o[k] * inv, 0.f) & 0xffffu);
}

}  // namespace

namespace pkv_latent {
uint32_t take_status()
{
    uint32_t v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_status, sizeof v) != cudaSuccess) return 0;
    if (v) cudaMemcpyToSymbol(g_status, &z, sizeof z);
    return v;
}
}  // namespace pkv_latent

extern "C" {

size_t paged_latent_attention_workspace_size(int32_t num_seqs, int32_t total_q_tokens, int32_t num_heads,
                                             int32_t max_blocks_per_seq)
{
    (void)num_seqs, (void)total_q_tokens, (void)num_heads, (void)max_blocks_per_seq;
    return 0;
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
    if (num_heads > PAGEDKV_LATENT_MAX_HEADS || max_blocks_per_seq > INT32_MAX / BS || num_blocks > INT32_MAX / BS)
        return KV_ERR_UNSUPPORTED;
    if (!out || !q || !context_lens || !cache || !block_tables) return KV_ERR_INVALID;
    if (!cu_q_lens && total_q_tokens != num_seqs) return KV_ERR_INVALID;
    if (!(scale > 0.f) || !std::isfinite(scale)) return KV_ERR_INVALID;
    if (!pkv_host::aligned(out, 16) || !pkv_host::aligned(q, 16) || !pkv_host::aligned(cache, 16) ||
        !pkv_host::aligned(block_tables, 4) || !pkv_host::aligned(context_lens, 4) ||
        (cu_q_lens && !pkv_host::aligned(cu_q_lens, 4)))
        return KV_ERR_INVALID;
    const size_t need =
        paged_latent_attention_workspace_size(num_seqs, total_q_tokens, num_heads, max_blocks_per_seq);
    if (need && (!workspace || workspace_bytes < need || !pkv_host::aligned(workspace, 256))) return KV_ERR_INVALID;
    const LatentParams p = {static_cast<uint16_t *>(out), static_cast<const uint16_t *>(q),
                            static_cast<const uint16_t *>(cache), cu_q_lens, context_lens, block_tables, num_seqs,
                            total_q_tokens, num_heads, max_blocks_per_seq, num_blocks, scale * LOG2E};
    const long long warps = (long long)total_q_tokens * num_heads;
    if ((warps + 7) / 8 > INT32_MAX) return KV_ERR_UNSUPPORTED;
    latent_simple_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

}  // extern "C"
