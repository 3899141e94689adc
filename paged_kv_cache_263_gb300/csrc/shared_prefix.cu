// shared_prefix.cu -- decode attention for a batch whose sequences share prefixes
// (sm_103a).
//
//   out[r][h] = sum_t p_t v_t,  p = softmax_t(scale x q[r][h] . k_t)
// over the keys of a row's whole context: its group's prefix, then its own tail.
#include "shared_prefix.cuh"
#include "trace.h"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

namespace {

__device__ uint32_t g_status;

using namespace pkv;

constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ void flag(uint32_t bits) { atomicOr(&g_status, bits); }

struct SharedParams {
    SharedBatch b;
    __nv_bfloat16 *out;
    const uint16_t *q;
    const void *k_cache, *v_cache;
    const int32_t *block_tables;
    const float *k_scale, *v_scale;
    int hq, hkv, num_blocks;
    float scale_log2;
};

template <bool FP8>
__device__ __forceinline__ float4 load4(const void *cache, size_t at)
{
    if constexpr (FP8) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(cache) + at);
        const uint32_t a = e4m3x2_to_f16x2(w & 0xffffu), b = e4m3x2_to_f16x2(w >> 16);
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
        return make_float4(x.x, x.y, y.x, y.y);
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(cache) + at);
        return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    }
}

// One CTA of 4 warps a (sequence, head): every row of the sequence in turn, keys
// t = warp, warp + 4, ..., four dims a lane.
template <bool FP8>
__global__ void __launch_bounds__(128) shared_prefix_kernel(const SharedParams p)
{
    __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
    const int s = blockIdx.x, h = blockIdx.y, g = h / (p.hq / p.hkv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SharedSeq w = shared_seq(p.b, s);
    if (w.state == SEQ_BAD) {
        if (h == 0 && threadIdx.x == 0) flag(ST_BAD_LEN);
        return;
    }
    const float ks = FP8 ? p.k_scale[g] : 1.f, vs = FP8 ? p.v_scale[g] : 1.f;
    for (int i = 0; i < w.n; ++i) {
        __nv_bfloat16 *out = p.out + ((size_t)(w.row0 + i) * p.hq + h) * D;
        if (w.state == SEQ_EMPTY) {
            out[threadIdx.x] = __float2bfloat16(0.f);
            continue;
        }
        const uint2 qw = *reinterpret_cast<const uint2 *>(p.q + ((size_t)(w.row0 + i) * p.hq + h) * D + 4 * lane);
        const float4 q = make_float4(bf16_lo(qw.x), bf16_hi(qw.x), bf16_lo(qw.y), bf16_hi(qw.y));
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const int keys = w.L - w.n + i + 1;
        for (int t = warp; t < keys; t += 4) {
            const int row = t < w.P ? w.first : s;
            const int id = __ldg(p.block_tables + (size_t)row * p.b.max_blocks + t / BS);
            if (id < 0 || id >= p.num_blocks) {
                if (lane == 0) flag(ST_BAD_BLOCK);
                continue;
            }
            const size_t at = (((size_t)id * p.hkv + g) * BS + t % BS) * D + 4 * lane;
            const float4 k = load4<FP8>(p.k_cache, at), v = load4<FP8>(p.v_cache, at);
            float x = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
            for (int o2 = 16; o2 > 0; o2 >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o2);
            x *= p.scale_log2 * ks;
            const float mn = fmaxf(m, x), r = mn == -INFINITY ? 0.f : mn;
            const float a = ex2(m - r), e = ex2(x - r);
            m = mn;
            l = l * a + e;
            o = make_float4(o.x * a + e * v.x, o.y * a + e * v.y, o.z * a + e * v.z, o.w * a + e * v.w);
        }
        if (lane == 0) {
            sm_m[warp] = m;
            sm_l[warp] = l;
        }
        *reinterpret_cast<float4 *>(&sm_o[warp][4 * lane]) = o;
        __syncthreads();
        const float M = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3])), R = M == -INFINITY ? 0.f : M;
        float ls = 0.f, os = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float f = ex2(sm_m[u] - R);
            ls += f * sm_l[u];
            os += f * sm_o[u][threadIdx.x];
        }
        out[threadIdx.x] = __float2bfloat16(ls == 0.f ? 0.f : os * vs / ls);
        __syncthreads();
    }
}

}  // namespace

namespace pkv_shared {
cudaError_t status_word(uint32_t **at) { return cudaGetSymbolAddress(reinterpret_cast<void **>(at), g_status); }
}  // namespace pkv_shared

extern "C" {

size_t paged_attention_shared_prefix_workspace_size(int32_t num_seqs, int32_t total_q_tokens, int32_t max_q_len,
                                                    int32_t num_groups, int32_t num_q_heads, int32_t num_kv_heads,
                                                    int32_t max_prefix_len, int32_t max_tail_len)
{
    (void)num_seqs, (void)total_q_tokens, (void)max_q_len, (void)num_groups, (void)num_q_heads, (void)num_kv_heads;
    (void)max_prefix_len, (void)max_tail_len;
    return 0;
}

kv_status paged_attention_shared_prefix(void *out, const void *q, const int32_t *cu_q_lens,
                                        const int32_t *context_lens, int32_t num_seqs, int32_t total_q_tokens,
                                        int32_t max_q_len, const int32_t *cu_groups, const int32_t *prefix_lens,
                                        int32_t num_groups, int32_t max_prefix_len, int32_t max_tail_len,
                                        const void *k_cache, const void *v_cache, const int32_t *block_tables,
                                        int32_t max_blocks_per_seq, int32_t num_q_heads, int32_t num_kv_heads,
                                        int32_t num_blocks, float scale, kv_dtype dtype, const float *k_scale,
                                        const float *v_scale, void *workspace, size_t workspace_bytes, void *stream)
{
    PKV_NVTX_RANGE("paged_attention_shared_prefix");
    if (num_seqs < 0 || total_q_tokens < 0 || num_groups < 0 || max_q_len < 1 || max_prefix_len < 0 || max_tail_len < 0 ||
        num_q_heads < 1 || num_kv_heads < 1 || num_blocks < 1 || max_blocks_per_seq < 1 || num_q_heads % num_kv_heads)
        return KV_ERR_INVALID;
    if (max_blocks_per_seq > INT32_MAX / BS) return KV_ERR_UNSUPPORTED;
    const int G = num_q_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8 && G != 16) return KV_ERR_UNSUPPORTED;
    if (dtype != KV_BF16 && dtype != KV_FP8_E4M3) return KV_ERR_UNSUPPORTED;
    if (dtype == KV_FP8_E4M3 && (!k_scale || !v_scale)) return KV_ERR_INVALID;
    if (!(scale > 0.f) || !(scale < INFINITY) || num_seqs > 65535 || num_kv_heads > 65535) return KV_ERR_INVALID;
    if (!cu_q_lens && (total_q_tokens != num_seqs || max_q_len != 1)) return KV_ERR_INVALID;
    if (num_groups > 65535) return KV_ERR_INVALID;
    if (num_seqs == 0 || total_q_tokens == 0) return KV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens ||
        (num_groups > 0 && (!cu_groups || !prefix_lens)))
        return KV_ERR_INVALID;
    if ((int64_t)num_blocks * num_kv_heads * BS > INT32_MAX) return KV_ERR_UNSUPPORTED;
    for (const void *x : {static_cast<const void *>(out), q, k_cache, v_cache})
        if (!pkv_host::aligned(x, 16)) return KV_ERR_INVALID;
    for (const int32_t *x : {cu_q_lens, context_lens, cu_groups, prefix_lens, block_tables})
        if (!pkv_host::aligned(x, 4)) return KV_ERR_INVALID;
    SharedParams p{};
    p.b = {cu_groups, prefix_lens, cu_q_lens, context_lens, num_groups, num_seqs, total_q_tokens, max_q_len,
           max_prefix_len / BS * BS, max_tail_len, max_blocks_per_seq};
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.q = static_cast<const uint16_t *>(q);
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * LOG2E;
    (void)workspace, (void)workspace_bytes;
    const dim3 grid(num_seqs, num_q_heads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == KV_BF16) shared_prefix_kernel<false><<<grid, 128, 0, st>>>(p);
    else shared_prefix_kernel<true><<<grid, 128, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

}  // extern "C"
