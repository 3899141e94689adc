// shared_prefix.cu -- decode attention for a batch whose sequences share prefixes
// (sm_103a).
//
//   out[r][h] = sum_t p_t v_t,  p = softmax_t(scale x q[r][h] . k_t)
// over the keys of a row's whole context: its group's prefix, then its own tail.
#include "shared_prefix.h"
#include "trace.h"

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

namespace {

__device__ uint32_t g_status;

using namespace pkv;

constexpr float LOG2E = 1.4426950408889634f;

struct MergeParams {
    SharedBatch b;
    __nv_bfloat16 *out;
    const float *part_o, *part_ml;
    int hq, prefix_splits, splits;         // splits: of prefix and tail together
    int tile_keys, prefix_tiles, tail_part_blocks, fine_from, fine_blocks, whole;
};

// Joins a row's parts, those of its group's prefix and those of its own tail, by the
// log-sum-exp rule in a fixed order: one warp a (row, head), four dims a lane.
constexpr int MERGE_WARPS = 8;
__global__ void __launch_bounds__(32 * MERGE_WARPS) shared_merge_kernel(const MergeParams p)
{
    const int row = blockIdx.x, h = blockIdx.y * MERGE_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    // (what describes the batch was written before the kernels of the parts began)
    const int s = p.b.cu_q_lens ? last_at_most(p.b.cu_q_lens, p.b.num_seqs, row, lane) : row;
    const SharedSeq w = shared_seq(p.b, s, lane);
    griddep_wait();
    griddep_launch_dependents();
    if (h >= p.hq || w.state == SEQ_BAD || row < w.row0 || row >= w.row0 + w.n) return;
    uint2 *out = reinterpret_cast<uint2 *>(p.out + ((size_t)row * p.hq + h) * D) + lane;
    if (w.state == SEQ_EMPTY) {
        *out = make_uint2(0u, 0u);
        return;
    }
    const int P = p.whole ? 0 : w.P;          // keys that have parts of their own
    const int KT = (P + p.tile_keys - 1) / p.tile_keys, np = KT ? (KT + p.prefix_tiles - 1) / p.prefix_tiles : 0;
    const int blocks = (w.L - P + BS - 1) / BS, part = s < p.fine_from ? p.tail_part_blocks : p.fine_blocks;
    const int nt = (blocks + part - 1) / part;
    const size_t base = ((size_t)row * p.hq + h) * p.splits;
    auto at = [&](int i) { return base + (i < np ? i : p.prefix_splits + i - np); };
    const int n = np + nt;
    // the first 32 parts' (max, sum), a part a lane, and the first parts' rows are asked
    // for together, before anything depends on them
    constexpr int AHEAD = 8;
    float2 e0 = make_float2(-INFINITY, 0.f);
    if (lane < n) e0 = *reinterpret_cast<const float2 *>(p.part_ml + 2 * at(lane));
    float4 v[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
        if (u < n) v[u] = reinterpret_cast<const float4 *>(p.part_o + at(u) * D)[lane];
    float M = e0.x;
    for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, p.part_ml[2 * at(i)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    // (no finite maximum: a row whose sums are not numbers stays one)
    const float R = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
        if (i0 > 0) e0 = i0 + lane < n ? *reinterpret_cast<const float2 *>(p.part_ml + 2 * at(i0 + lane)) : make_float2(-INFINITY, 0.f);
        const float weight = ex2(e0.x - R), part = weight * e0.y;
        for (int k0 = 0; k0 < min(32, n - i0); k0 += AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int i = i0 + k0 + u;
                const float f = __shfl_sync(0xffffffffu, weight, k0 + u), l = __shfl_sync(0xffffffffu, part, k0 + u);
                if (i < n) {
                    sum += l;
                    acc.x += f * v[u].x;
                    acc.y += f * v[u].y;
                    acc.z += f * v[u].z;
                    acc.w += f * v[u].w;
                }
                if (i + AHEAD < n) v[u] = reinterpret_cast<const float4 *>(p.part_o + at(i + AHEAD) * D)[lane];
            }
        }
    }
    // (every row sees a key: a sum of 0 is scores that are all -inf, whose softmax is NaN)
    const float inv = 1.f / sum;
    *out = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

// How a call is done, from its sizes and bounds: the way that these costs say is the
// shortest, in us of the 152 SMs, for blocks of 16 keys.
//
// whole: one kernel attends whole contexts, at most 16 rows x heads an item (a set of a
// sequence's rows), and reads a prefix once a set, from L2 where it fits.  A set takes
// SET_US, a block FIRST_US where it comes from memory and AGAIN_US for each further set
// that reads it (fp8: FIRST8_US, AGAIN8_US).
// apart: the prefixes in the chunk kernel's tiles, the tails beside it as above.  A block
// of a prefix takes TILE_US for a query item (256 rows x heads; BIG_US for 128 where a
// group has no more, over a bf16 cache; fp8 TILE8_US): more than the tiles' own time, as
// the items and the prefixes are unequal.
// joined: the chunk kernel takes the tails as well, TAIL_ITEM_US an item and less a block
// than for prefixes, as each tail is read once.  (TAIL_TILE_US and its like are by the block,
// of whole calls.  The lengths of joined parts go by costs of their own, JOIN_TILE_US and
// JOIN_ITEM_US in prefill.cu, by the tile and fitted to calls that differ in those lengths
// alone: there an item is 4 us and a tile of four blocks 1.03, here 7.2 and 0.73, as a
// whole call's items hold what its start and uneven end take.)  Only for rows x heads of a sequence that are
// more than 16: at 16 it lost (32 sequences x 4 rows: 62.5 us against 52.5).
// ROOT_US: the last parts and the merge of long contexts, which are cut into about the
// root of their blocks.
//
// Measured on 180 drawn batches, each way forced in turn: the costs' choice takes 1 % more
// than the best way (2 % when fitted on the other half); rules by sequences a group and keys
// of prefix, with joined for all wide rows, took 3 % more for narrow rows and 16 % for wide
// ones.  Some of them, us (rows x heads of a sequence):
//                                                        whole   apart   joined
//   152 sequences x 32, prefixes to 600, tails to 200    27.6    47.3    47.2
//   51 x 56, one prefix of 12K, tails to 180, fp8        205     45.2    62.1
//   49 x 56, tails of 7K to 11K                          205     243     125
//   16 groups of 2 x 4, 24,576 of prefix                 236     263
//   8 groups of 16 x 4, 1,500 of prefix                  17.7    15.9
//
// Whole contexts are cut into the number of parts whose cost is the least, in us: what an
// item takes to begin and to end, ITEM_US times the items a CTA; what the last items
// take alone, BLOCK_US a block; a row's parts in the merge, PART_US each; the merge
// itself, and a counter of items where there are more than CTAs.  (Blocks a part,
// measured, us; 8 items a part, 1,094 blocks: 16 26.4, 28 25.8, 36 19.2, 64 20.6, 100 25.6;
// 31 of 464: 16 17.8, 24 14.3, 36 14.2, 64 16.8; 672 of 91, fp8: 46 46.0, 91 41.2; 252 of
// 1,056, fp8: 36 136.9, 64 128.5, 118 128.4.  Over 46 drawn batches the choice is 2 % off
// the best of 12 lengths, and a fixed one of 16 blocks or two items a CTA 7 %.)
//
// Tails beside the prefixes: parts of TAIL_ROOT times the root of their blocks, or of
// TAIL_WANT of what gives TAIL_CTAS items where that is more, and of at most 256 (75 drawn
// batches with 13 lengths each: 2 % off the best length; 48 sequences of 100 to 2,500 tokens
// beside two prefixes, fp8: 49.2 us with 24 blocks, 45.4 with 40, 45.1 with 100, 45.0 as
// chosen; 64 of 20 to 1,000 beside one, bf16: 86.6, 85.2, 81.1 and 81.0; 128 of 1,024 to
// 16,384: 661, 661, 653 and 645).  The last fifth of the sequences has parts of half the
// length, so that the last items are short (the first of these batches 47.1 us without, the
// last 651, 32 sequences x 4 rows 44.0 for 43.5; a third or half of the sequences gain less;
// contexts that are one part lose 1 us by it, whole contexts up to 4 us of 15).
//
// All of these were fitted to batches whose bounds were their own longest prefix and tail,
// with up to 256 sequences.
//
constexpr int64_t TAIL_COLS = 16, TAIL_CTAS = 2 * 3 * 152;
constexpr double TAIL_ROOT = 2.6, TAIL_WANT = 0.9;
constexpr double SET_US = 1.5, FIRST_US = 0.133, AGAIN_US = 0.077, FIRST8_US = 0.153, AGAIN8_US = 0.055;
constexpr double TILE_US = 0.295, BIG_US = 0.215, TILE8_US = 0.32;
constexpr double TAIL_ITEM_US = 7.2, TAIL_TILE_US = 0.183, TAIL_BIG_US = 0.158, TAIL_TILE8_US = 0.227;
constexpr double WHOLE_START_US = 6, APART_START_US = 11.7, JOINED_START_US = 9.2, ROOT_US = 0.157;
constexpr double ITEM_US = 1.5, BLOCK_US = 0.15, PART_US = 0.15, MERGE_US = 4, COUNTER_US = 1.2;

void choose(SharedCall &c, int32_t max_tail_len)
{
    const int G = c.hq / c.hkv;
    const int64_t groups = c.b.num_groups, rows = c.b.total_rows;
    const double seqs = std::max(1, c.b.num_seqs), sms = 152;
    const double P = groups ? (double)(c.b.max_prefix / BS) : 0, T = ((double)max_tail_len + BS - 1) / BS;
    const double mean = std::max(1.0, (double)rows / seqs);          // rows of a sequence
    const double sets = c.mean_sets;
    const double first = c.fp8 ? FIRST8_US : FIRST_US, again = c.fp8 ? AGAIN8_US : AGAIN_US;
    const double tails = seqs * c.hkv * (SET_US * sets + (first + (sets - 1) * again) * T) / sms;
    const double readers = std::min((double)groups, seqs);
    auto big = [&](bool joined) {
        const double of = P > 0 ? (double)groups : seqs;
        return !c.fp8 && (double)rows * G <= 128 * of && (!joined || (int64_t)c.b.max_q_len * G <= 128);
    };
    auto prefix = [&](bool is_big) {
        if (P == 0) return 0.0;
        const double items = std::ceil((double)rows / groups / ((is_big ? 128 : 256) / G));
        return groups * items * c.hkv * P * (c.fp8 ? TILE8_US : is_big ? BIG_US : TILE_US) / sms;
    };
    const double whole = WHOLE_START_US + tails + c.hkv * P * (first * readers + again * (seqs * sets - readers)) / sms +
                         ROOT_US * std::sqrt(P + T);
    const double apart = P > 0 ? APART_START_US + prefix(big(false)) + tails + ROOT_US * std::sqrt(T) : INFINITY;
    double joined = INFINITY;
    if (c.b.max_q_len > 1 && (int64_t)c.b.max_q_len * G > TAIL_COLS) {
        const bool is_big = big(true);
        const double items = seqs * std::ceil(mean / ((is_big ? 128 : 256) / G)) * c.hkv;
        joined = JOINED_START_US + prefix(is_big) +
                 items * (TAIL_ITEM_US + T * (c.fp8 ? TAIL_TILE8_US : is_big ? TAIL_BIG_US : TAIL_TILE_US)) / sms;
    }
    c.joined = joined < std::min(whole, apart);
    c.whole = !c.joined && whole <= apart;
}

// A call's partial results are at most those that PART_BYTES hold, or two parts a row where
// that is more: so the workspace's size grows with every argument, and the one for the
// largest batch serves all.  No drawn batch with bounds of its own has more (2,333, up to
// 256 sequences; 24 with bounds 16 times its tails).
constexpr int64_t PART_EACH = D * 4 + 8, PART_BYTES = 128 << 20;
int64_t room_for(const SharedCall &c)       // partial results of one row and head
{
    return std::max<int64_t>(2 * (int64_t)c.b.total_rows * c.hq, PART_BYTES / PART_EACH);
}
int64_t whole_parts(int64_t blocks) { return std::min<int64_t>(256, (blocks + 11) / 12); }
// the most parts that a row has with these bounds or lower ones, whichever way the call goes
// (plan below and plan_prefixes)
int64_t parts_at_most(const SharedCall &c, int32_t max_tail_len)
{
    const int64_t P = c.b.num_groups > 0 ? c.b.max_prefix / BS : 0, T = ((int64_t)max_tail_len + BS - 1) / BS;
    const int64_t tiles = std::min<int64_t>(128, (P * BS + 63) / 64);
    int64_t most = std::max<int64_t>(1, whole_parts(P + T));
    if (P > 0) {
        const int64_t cut = std::max<int64_t>({1, (int64_t)((double)T / (TAIL_ROOT * std::sqrt(std::max(1.0, (double)T)))),
                                               (T + 255) / 256});
        most = std::max(most, tiles + (cut > 1 ? 2 * cut : 1));
    }
    if (c.b.max_q_len > 1 && (int64_t)c.b.max_q_len * (c.hq / c.hkv) > TAIL_COLS)
        most = std::max(most, tiles + std::max<int64_t>(1, std::min<int64_t>(128, ((int64_t)max_tail_len + 63) / 64)));
    return most;
}

void plan(SharedCall &c, int32_t max_tail_len)
{
    const int64_t groups = c.b.num_groups;
    c.most_parts = (int)std::min<int64_t>(room_for(c) / ((int64_t)c.b.total_rows * c.hq), INT32_MAX);
    c.set_rows = (int)(TAIL_COLS / (c.hq / c.hkv));
    c.sets = (c.b.max_q_len - 1) / c.set_rows + 1;
    c.mean_sets = std::ceil(std::max(1.0, (double)c.b.total_rows / std::max(1, c.b.num_seqs)) / c.set_rows);
    choose(c, max_tail_len);
    c.fine_from = INT32_MAX;
    c.fine_blocks = 1;
    c.prefix_splits = 0;
    c.prefix_items = c.tail_items = 0;
    if (!c.whole) pkv_prefill::plan_prefixes(c, max_tail_len);
    if (c.joined) return;
    const int64_t keys = (int64_t)max_tail_len + (c.whole && groups ? c.b.max_prefix : 0);
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((keys + BS - 1) / BS, INT32_MAX / BS));
    if (c.whole) {
        const double each = (double)c.b.num_seqs * c.hkv * c.mean_sets;
        const double ctas = (int64_t)c.b.max_q_len * (c.hq / c.hkv) > 8 ? 2 * 152 : 3 * 152;
        const int64_t most = std::min<int64_t>(c.most_parts, whole_parts(blocks));
        double best = 0;
        for (int64_t n = 1; n <= most; n += 1 + n / 16) {
            const double us = ITEM_US * n * each / ctas + BLOCK_US * (double)((blocks + n - 1) / n) +
                              PART_US * (double)n + (n > 1 ? MERGE_US + (n * each > ctas ? COUNTER_US : 0) : 0);
            if (n == 1 || us < best) {
                best = us;
                c.tail_splits = (int)n;
            }
        }
    } else {
        const double want = (double)blocks * c.b.num_seqs * c.hkv / TAIL_CTAS;
        const double part = std::max(TAIL_ROOT * std::sqrt((double)blocks), TAIL_WANT * want);
        const int64_t cut = std::max<int64_t>({1, (int64_t)((double)blocks / part), (blocks + 255) / 256});
        // (twice as many with the shorter parts at the end)
        c.tail_splits = (int)std::min<int64_t>(cut, std::max(1, (c.most_parts - c.prefix_splits) / 2));
    }
    c.tail_part_blocks = (int)((blocks + c.tail_splits - 1) / c.tail_splits);
    if (!c.whole && c.tail_splits > 1) {
        c.fine_from = (int)((int64_t)c.b.num_seqs * 4 / 5);
        c.fine_blocks = (c.tail_part_blocks + 1) / 2;
        c.tail_splits = (int)((blocks + c.fine_blocks - 1) / c.fine_blocks);
    }
}

size_t up(size_t n) { return (n + 255) & ~size_t(255); }
// (none where the only part is the output)
size_t part_o_bytes(const SharedCall &c)
{
    if (shared_parts(c) == 1) return 0;
    return up((size_t)c.b.total_rows * c.hq * shared_parts(c) * D * sizeof(float));
}
size_t part_ml_bytes(const SharedCall &c)
{
    if (shared_parts(c) == 1) return 0;
    return up((size_t)c.b.total_rows * c.hq * shared_parts(c) * 2 * sizeof(float));
}

// what the caller provides: room for the parts of this call's plan and of any smaller call's
size_t scratch_bytes(const SharedCall &c, int32_t max_tail_len)
{
    const int64_t parts = parts_at_most(c, max_tail_len), rh = (int64_t)c.b.total_rows * c.hq;
    if (parts == 1) return 0;
    const int64_t n = rh > INT64_MAX / parts ? room_for(c) : std::min(rh * parts, room_for(c));
    return up((size_t)n * D * sizeof(float)) + up((size_t)n * 2 * sizeof(float)) + 256;      // and the counter
}

// the description that sizes and bounds alone make (false: sizes that no call takes)
bool describe(SharedCall &c, int32_t num_seqs, int32_t total_q_tokens, int32_t max_q_len, int32_t num_groups,
              int32_t num_q_heads, int32_t num_kv_heads, int32_t max_prefix_len, int32_t max_tail_len, bool fp8)
{
    if (num_seqs < 1 || total_q_tokens < 1 || max_q_len < 1 || num_groups < 0 || num_q_heads < 1 || num_kv_heads < 1 ||
        max_prefix_len < 0 || max_tail_len < 0 || num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > 16 ||
        num_q_heads > 65535 * MERGE_WARPS)
        return false;
    c.b.num_seqs = num_seqs;
    c.b.total_rows = total_q_tokens;
    c.b.max_q_len = max_q_len;
    c.b.num_groups = num_groups;
    c.b.max_prefix = max_prefix_len / BS * BS;
    c.hq = num_q_heads;
    c.hkv = num_kv_heads;
    c.fp8 = fp8;
    return true;
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
    SharedCall c{};
    if (!describe(c, num_seqs, total_q_tokens, max_q_len, num_groups, num_q_heads, num_kv_heads, max_prefix_len,
                  max_tail_len, false))
        return 0;
    return scratch_bytes(c, max_tail_len);
}

int32_t paged_attention_shared_prefix_way(int32_t num_seqs, int32_t total_q_tokens, int32_t max_q_len, int32_t num_groups,
                                          int32_t num_q_heads, int32_t num_kv_heads, int32_t max_prefix_len,
                                          int32_t max_tail_len, kv_dtype dtype)
{
    SharedCall c{};
    if ((dtype != KV_BF16 && dtype != KV_FP8_E4M3) ||
        !describe(c, num_seqs, total_q_tokens, max_q_len, num_groups, num_q_heads, num_kv_heads, max_prefix_len,
                  max_tail_len, dtype == KV_FP8_E4M3))
        return -1;
    plan(c, max_tail_len);
    return c.whole ? 0 : c.joined ? 2 : 1;
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
    // (keys and a tile more are counted in 32 bits)
    if (max_blocks_per_seq > (INT32_MAX - 255) / BS || num_q_heads > 65535 * MERGE_WARPS) return KV_ERR_UNSUPPORTED;
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
    SharedCall c{};
    c.b = {cu_groups, prefix_lens, cu_q_lens, context_lens, num_groups, num_seqs, total_q_tokens, max_q_len,
           max_prefix_len / BS * BS, max_tail_len, max_blocks_per_seq};
    c.out = out;
    c.q = static_cast<const uint16_t *>(q);
    c.k_cache = k_cache;
    c.v_cache = v_cache;
    c.block_tables = block_tables;
    c.k_scale = k_scale;
    c.v_scale = v_scale;
    c.hq = num_q_heads;
    c.hkv = num_kv_heads;
    c.num_blocks = num_blocks;
    c.fp8 = dtype == KV_FP8_E4M3;
    c.scale_log2 = scale * LOG2E;
    plan(c, max_tail_len);
    // (32 groups that claim all rows, as malformed data may, still count their items in 32 bits)
    if (c.prefix_items > INT32_MAX / 64 || c.tail_items > INT32_MAX / 64) return KV_ERR_UNSUPPORTED;
    if (c.joined && ((int64_t)max_q_len * G / 128 + 1) * num_kv_heads * c.tail_splits > INT32_MAX / 64)
        return KV_ERR_UNSUPPORTED;
    // (and 32 sequences in the tails' kernel, of which each may claim all rows)
    if ((int64_t)max_q_len * G > INT32_MAX / 32 || tail_kernel_items(c) > INT32_MAX / 2 ||
        (int64_t)std::min(max_q_len, total_q_tokens) / c.set_rows + 1 > INT32_MAX / 64 / num_kv_heads / c.tail_splits)
        return KV_ERR_UNSUPPORTED;
    // (the plan and the workspace's size go by the bounds as given; no length passes what a
    // table row holds)
    const size_t need = scratch_bytes(c, max_tail_len);
    c.b.max_prefix = std::min(c.b.max_prefix, max_blocks_per_seq * BS);
    c.b.max_tail = std::min(c.b.max_tail, max_blocks_per_seq * BS);
    const size_t o_bytes = part_o_bytes(c);
    if (need && (!workspace || !pkv_host::aligned(workspace, 256) || workspace_bytes < need)) return KV_ERR_INVALID;
    c.part_o = static_cast<float *>(workspace);
    c.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + o_bytes);
    c.counter = reinterpret_cast<int *>(static_cast<uint8_t *>(workspace) + o_bytes + part_ml_bytes(c));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool prefixes = c.prefix_splits > 0 || c.joined;
    if (prefixes && pkv_prefill::launch_prefixes(c, st) != cudaSuccess) return KV_ERR_CUDA;
    if (!c.joined && pkv_shared_tail::launch_tails(c, prefixes, st) != cudaSuccess) return KV_ERR_CUDA;
    if (!o_bytes) return KV_OK;
    const MergeParams m = {c.b, static_cast<__nv_bfloat16 *>(out), c.part_o, c.part_ml, num_q_heads, c.prefix_splits,
                           shared_parts(c), c.big ? 128 : 64, c.prefix_tiles, c.tail_part_blocks, c.fine_from,
                           c.fine_blocks, c.whole ? 1 : 0};
    const dim3 grid(total_q_tokens, (num_q_heads + MERGE_WARPS - 1) / MERGE_WARPS);
    return pkv_host::launch_ex(shared_merge_kernel, grid, dim3(32 * MERGE_WARPS), 0, st, true, m) == cudaSuccess
               ? KV_OK : KV_ERR_CUDA;
}

}  // extern "C"
