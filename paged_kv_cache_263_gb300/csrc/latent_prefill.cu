// latent_prefill.cu -- attention over expanded latents, for prompts (sm_103a).
//
// kv[t][h] holds head h's key part (128, expanded from the token's latent) and
// value (128); the rotary key k_rope[t] (64) is shared by all heads:
//   out[r][h] = sum_t p_t kv[t][h][128:],
//   p = softmax_t(scale * (q[r][h][:128] . kv[t][h][:128] + q[r][h][128:] . k_rope[t]))
// over the keys t <= nk - nq + i that row i of a sequence's nq rows sees.
#include "common.cuh"
#include "trace.h"

#include <algorithm>
#include <cmath>

namespace {

__device__ uint32_t g_status;

using namespace pkv;

constexpr float LOG2E = 1.4426950408889634f;

struct ExpandedParams {
    uint16_t *out;
    const uint16_t *q, *kv, *rope;
    const int32_t *cu_q, *cu_k;
    int64_t rope_stride;
    int num_seqs, rows, keys, heads;
    float scale_log2;
};

__device__ __forceinline__ void flag(uint32_t bits) { atomicOr(&g_status, bits); }

// One warp per (row, head): lane l holds dims l, l + 32, ... of q and of the sum.
__global__ void __launch_bounds__(256) expanded_simple_kernel(const ExpandedParams p)
{
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= (long long)p.rows * p.heads) return;
    const int row = (int)(w / p.heads), h = (int)(w % p.heads);
    int s = -1, a = 0, n = 0;
    for (int i = 0; i < p.num_seqs; ++i)
        if (p.cu_q[i] <= row && row < p.cu_q[i + 1]) {
            s = i;
            a = p.cu_q[i];
            n = p.cu_q[i + 1] - a;
            break;
        }
    if (s < 0) return;
    const int k0 = p.cu_k[s], nk = p.cu_k[s + 1] - k0;
    if (a < 0 || a + n > p.rows || k0 < 0 || nk < 0 || k0 + nk > p.keys) {
        if (lane == 0) flag(ST_BAD_LEN);
        return;
    }
    const int last = nk - n + (row - a);
    float q[6], o[4], m = -INFINITY, l = 0.f;
    for (int k = 0; k < 6; ++k) q[k] = __uint_as_float((uint32_t)p.q[w * (D + ROPE) + lane + 32 * k] << 16);
    for (int k = 0; k < 4; ++k) o[k] = 0.f;
    for (int t = 0; t <= last; ++t) {
        const uint16_t *x = p.kv + ((size_t)(k0 + t) * p.heads + h) * (2 * D);
        const uint16_t *r = p.rope + (k0 + t) * p.rope_stride;
        float d = 0.f;
        for (int k = 0; k < 4; ++k) d += q[k] * __uint_as_float((uint32_t)x[lane + 32 * k] << 16);
        for (int k = 0; k < 2; ++k) d += q[4 + k] * __uint_as_float((uint32_t)r[lane + 32 * k] << 16);
        for (int b = 16; b > 0; b >>= 1) d += __shfl_xor_sync(0xffffffffu, d, b);
        d *= p.scale_log2;
        const float mn = fmaxf(m, d), c = ex2(m - mn), e = ex2(d - mn);
        l = l * c + e;
        for (int k = 0; k < 4; ++k) o[k] = o[k] * c + e * __uint_as_float((uint32_t)x[D + lane + 32 * k] << 16);
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int k = 0; k < 4; ++k) p.out[w * D + lane + 32 * k] = (uint16_t)(pack_bf16(o[k] * inv, 0.f) & 0xffffu);
}

}  // namespace

namespace pkv_latent_prefill {
uint32_t take_status()
{
    uint32_t v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_status, sizeof v) != cudaSuccess) return 0;
    if (v) cudaMemcpyToSymbol(g_status, &z, sizeof z);
    return v;
}
}  // namespace pkv_latent_prefill

extern "C" {

size_t latent_prefill_attention_workspace_size(int32_t num_seqs, int32_t total_q_tokens, int32_t num_heads)
{
    (void)num_seqs, (void)total_q_tokens, (void)num_heads;
    return 0;
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
    const ExpandedParams p = {static_cast<uint16_t *>(out), static_cast<const uint16_t *>(q),
                              static_cast<const uint16_t *>(kv), static_cast<const uint16_t *>(k_rope), cu_q_lens,
                              cu_k_lens, k_rope_stride, num_seqs, total_q_tokens, total_k_tokens, num_heads,
                              scale * LOG2E};
    const long long warps = (long long)total_q_tokens * num_heads;
    if ((warps + 7) / 8 > INT32_MAX) return KV_ERR_UNSUPPORTED;
    expanded_simple_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

}  // extern "C"
