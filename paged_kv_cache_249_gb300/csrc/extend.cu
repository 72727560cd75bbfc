// extend.cu -- the calls for several new tokens per sequence (extend and
// tree attention): host-side checks, the split over the context, and the
// log-sum-exp pass that joins a split row's parts.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "extend_common.cuh"

namespace pkv {
namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

constexpr int kExtMinPart = 256, kExtMinPartFma = 128;

struct alignas(64) MapPair {
    CUtensorMap k, v;
};

// Automatic split: cut the keys of every tile into parts, of at least kExtMinPart
// (kExtMinPartFma on the CUDA cores), until the launch has about this many items if
// all sequences are as long as the longest (a batch usually holds shorter ones).
// Where two CTAs share an SM one's start and end hide behind the other, so more and
// shorter items are taken there.  Measured (us, by part length; "auto" is what these
// rules take):
//   tensor cores                      512   1024   2048   4096   8192   none   auto
//   32 trees of up to 32 nodes over
//     512-8192                        180    138    115    103    120    108    102
//   2 of up to 64 over 32768 and
//     98304 (256-row tiles)           637    410    282    242    219   1071    213
//   CUDA cores                         64    128    256    512   1024   none   auto
//   3 sequences of 33-257 tokens over
//     up to 500 more, head_dim 64    35.6   42.9   51.6   78.3   72.9   72.2   42.6
//   one of 512 tokens, head_dim 128  81.1   62.9   94.1    117    117    117   62.4
//   64 single tokens over 100-2000,
//     head_dim 64 (16-row tiles)     95.8   69.3   64.8   62.1    106    163   62.1
// (Parts of 64 would serve the first of the last three and cost the others.)
int tile_count(long long num_tokens, int num_seqs, int group, int rows) {
    return (int)(num_tokens * group / rows) + num_seqs;
}

long long wanted_items(int rows, int head_dim) {
    return rows == 128 ? (head_dim == 256 ? 300 : 520) : rows == 256 ? 400
                       : rows == 16 && head_dim == 64 ? 1200 : 600;
}

long long most_parts(int rows, long long range) {
    const int least = rows >= 128 ? kExtMinPart : kExtMinPartFma;
    return (range + least - 1) / least;
}

// Parts of the automatic split for a range of `range` keys.  Within the bounds
// above, as many as make the sum of two times least: a part's keys, one after
// another in a CTA, and the joining pass, which reads and writes every part of
// every row.  In us, measured on single CTAs and joining passes: D / 12800 a key,
// and 3 + D / 625000 for a part of a row.  (One sequence of 300 tokens 9.7 us
// unsplit, 16.9 in two parts; three of 100 over up to 1000 15.4 and 21.8.)  On the
// CUDA cores D / 1100 a key is not what a CTA alone takes (D / 610), but chooses
// well among the parts above.
int auto_parts(long long num_tokens, int num_seqs, int num_heads, int num_kv_heads, int rows,
               int head_dim, long long range) {
    const long long tiles =
        std::max<long long>(num_seqs, (num_tokens * (num_heads / num_kv_heads) + rows - 1) / rows);
    const long long want = wanted_items(rows, head_dim) / (tiles * num_kv_heads);
    const long long most = std::min(want, most_parts(rows, range));
    if (most < 2) return 1;
    const double keys = (double)range * head_dim / (rows >= 128 ? 12800. : 1100.);
    const double part = (double)num_tokens * num_heads * head_dim / 625000.;
    const long long parts = std::max(2ll, std::min(most, (long long)std::sqrt(keys / part)));
    return keys / parts + 3. + part * parts < keys ? (int)parts : 1;
}

size_t partial_bytes(long long rows, int head_dim, int parts, size_t *o_bytes) {
    const size_t n = (size_t)rows * parts;
    *o_bytes = round_up(n * head_dim * sizeof(float), 256);
    return *o_bytes + round_up(n * sizeof(float), 256);
}

// ------------------------------------------------------------------ combine
//
// Row (token, head) of a split call has parts p with normalised outputs o_p
// and log2-sum-exps e_p (-inf: the part saw no key, o_p is not written):
//   out = sum_p 2^(e_p - M) o_p / sum_p 2^(e_p - M),  M = max_p e_p.
// One warp per row of a tile; the tiles are those of the attention kernel, so
// rows that it skipped stay as they were.  Where query_starts are out of order or
// out of range, the attention's list of items may have no room for tiles that the
// search here finds (it has for those of the other wrong descriptions): their
// parts hold whatever the workspace held, so nothing is joined.
template <int D>
__global__ void __launch_bounds__(128) extend_combine_kernel(const ExtArgs a, int rows) {
    constexpr int PER = D / 32;
    griddep_launch();
    griddep_wait();
    const int kvh = blockIdx.x % a.num_kv_heads;
    bool wrong = false;
    if (a.num_seqs <= kExtScan)  // (with more, both find tiles by the same search)
        for (int s = threadIdx.x; s < a.num_seqs; s += 128) {
            const int q0 = __ldg(a.query_starts + s), q1 = __ldg(a.query_starts + s + 1);
            wrong |= q0 < 0 || q1 < q0 || q1 > a.num_tokens;
        }
    ExtTile t;
    const bool found = ext_find_tile(a, blockIdx.x / a.num_kv_heads, rows, t);
    if (__syncthreads_or(wrong) || !found) return;
    const int lane = threadIdx.x & 31;
    const int P = max(1, ext_num_parts(a, t));
    for (int r = blockIdx.y * 4 + threadIdx.x / 32; r < t.nrows; r += gridDim.y * 4) {
        const int row = t.row0 + r, tok = row / a.group;
        const size_t oh = (size_t)(t.q0 + tok) * a.num_heads + kvh * a.group + row - tok * a.group;
        const float *lse = a.ws_lse + oh * a.num_parts;
        const float *po = a.ws_o + oh * a.num_parts * D + lane * PER;
        float M = -CUDART_INF_F;
        for (int p = lane; p < P; p += 32) M = fmaxf(M, lse[p]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        const float ref = M == -CUDART_INF_F ? 0.f : M;
        float num[PER], den = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) num[j] = 0.f;
        for (int p = 0; p < P; ++p) {
            const float e = lse[p];
            if (e == -CUDART_INF_F) continue;
            const float w = exp2f(e - ref);  // NaN where the part's scores were
            den += w;
#pragma unroll
            for (int j = 0; j < PER; j += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(po + (size_t)p * D + j);
                num[j] = fmaf(w, v.x, num[j]), num[j + 1] = fmaf(w, v.y, num[j + 1]);
            }
        }
        const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
        for (int j = 0; j < PER; j += 2)
            store_out2(a.out, oh * D + lane * PER + j, num[j] * inv, num[j + 1] * inv, a.out_dtype);
    }
}

cudaError_t launch_combine(const ExtLaunch &L) {
    const dim3 grid((unsigned)(L.args.tiles * L.args.num_kv_heads),
                    (unsigned)((L.rows + 15) / 16));
    if (L.head_dim == 64)
        return launch_dependent(extend_combine_kernel<64>, grid, dim3(128), 0, L.stream, L.args, L.rows);
    if (L.head_dim == 128)
        return launch_dependent(extend_combine_kernel<128>, grid, dim3(128), 0, L.stream, L.args, L.rows);
    return launch_dependent(extend_combine_kernel<256>, grid, dim3(128), 0, L.stream, L.args, L.rows);
}

pkv_status extend_impl(const pkv_pool *pool, void *out, pkv_dtype out_dtype, const void *query,
                       int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                       const int32_t *block_tables, int max_blocks_per_seq,
                       const int32_t *context_lens, const int32_t *query_starts, int max_query_len,
                       int max_context_len, float scale, float softcap, int window,
                       const float *slopes, const int32_t *prefix_lens, bool tree,
                       const uint32_t *tree_mask, int mask_words, int partition_tokens,
                       void *workspace, size_t workspace_bytes, void *stream) {
    if (!pool || pool->magic != kPoolMagic || pool->layout != 0) return PKV_ERR_INVALID_ARG;
    if (num_tokens < 0 || num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        max_blocks_per_seq <= 0 || max_query_len < 0 || max_context_len < 0)
        return PKV_ERR_INVALID_ARG;
    if (num_kv_heads != pool->num_kv_heads || num_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    if (out_dtype != PKV_F32 && out_dtype != PKV_BF16 && out_dtype != PKV_F16)
        return PKV_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0)
        return PKV_ERR_INVALID_ARG;
    if (softcap > 0.f && !std::isfinite(4.f * scale / softcap)) return PKV_ERR_INVALID_ARG;
    if (tree && (mask_words < 0 || (long long)mask_words * 32 < max_query_len))
        return PKV_ERR_INVALID_ARG;
    if (partition_tokens < -1 || partition_tokens > kMaxPartitionTokens ||
        (partition_tokens > 0 && partition_tokens % pool->block_size != 0))
        return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0 || num_seqs == 0 || max_query_len == 0) return PKV_OK;
    if (!out || !query || !block_tables || !context_lens || !query_starts || (tree && !tree_mask))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(query, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(query_starts, 4) || !aligned(slopes, 4) ||
        !aligned(prefix_lens, 4) || !aligned(tree_mask, 4))
        return PKV_ERR_INVALID_ARG;
    const size_t values = (size_t)num_tokens * num_heads * pool->head_dim;
    const size_t q_bytes = values * (pool->dtype == PKV_F32 ? 4 : 2), out_bytes = values * (out_dtype == PKV_F32 ? 4 : 2);
    const uintptr_t q_at = reinterpret_cast<uintptr_t>(query), out_at = reinterpret_cast<uintptr_t>(out);
    if (q_at < out_at + out_bytes && out_at < q_at + q_bytes) return PKV_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if (group > kMaxGroup) return PKV_ERR_UNSUPPORTED;
    if (pool->dtype == PKV_F32 && pool->head_dim > 128) return PKV_ERR_UNSUPPORTED;
    int dev = 0;
    if (cuda_status(cudaGetDevice(&dev)) != PKV_OK) return PKV_ERR_CUDA;
    if (dev != pool->device) return PKV_ERR_INVALID_ARG;

    ExtLaunch L;
    ExtArgs &a = L.args;
    std::memset(&a, 0, sizeof(a));
    const long long table_cap = (long long)max_blocks_per_seq * pool->block_size;
    a.q = query;
    a.out = out;
    a.k_pool = pool->k_pool;
    a.v_pool = pool->v_pool;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_starts = query_starts;
    a.tree_mask = tree ? tree_mask : nullptr;
    a.mask_words = tree ? mask_words : 0;
    a.slopes = slopes;
    a.prefix_lens = prefix_lens;
    a.dev_error = pool->dev_error;
    a.num_tokens = num_tokens;
    a.num_seqs = num_seqs;
    a.max_query_len = max_query_len;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = group;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = pool->num_blocks;
    a.block_size = pool->block_size;
    while ((kExtRun << a.run_shift) < pool->block_size) ++a.run_shift;
    a.ctx_cap = (int)(table_cap < max_context_len ? table_cap : max_context_len);
    a.window = window;
    a.out_dtype = out_dtype;
    a.scale = scale;
    a.softcap = softcap;

    L.head_dim = pool->head_dim;
    L.stream = static_cast<cudaStream_t>(stream);
    L.device = dev;
    // On the tensor cores two CTAs of 128-row tiles share an SM, and one's start
    // and end run beside the other's tiles.  A CTA of 256 rows reads keys and
    // values half as often, which pays at head_dim 128 where sequences bring many
    // rows, ranges are long and scores need little work (us, 128 | 256 rows, 32
    // heads over 8 unless said): a prompt of 8192 tokens 400 | 377, of 16384 1550 |
    // 1378, 4 x 1024 tokens over 4000 271 | 251, 2 x 64 over 60000 with 64 heads
    // 233 | 222.  But 16 x 64 over 8000 142 | 155, 8 x 40 over 8000 with 64 heads
    // over 4 97 | 115, four prompts of 2048 155 | 157, 24 of 512 with 16 heads over
    // 16 65 | 77; and before both had rings of their own for K and V, capped
    // scores of 8192 tokens 565 | 623, head_dim 64 313 | 350.
    // On the CUDA cores a tile of 16 rows wastes less where no sequence brings more.
    const bool tc = pool->dtype != PKV_F32;
    const bool windowed = window > 0 && !prefix_lens && !tree;
    const long long seq_rows = (long long)max_query_len * group;
    const bool tall = pool->head_dim == 128 && seq_rows >= 512 && softcap == 0.f && !slopes &&
                      (windowed && window < a.ctx_cap ? window : a.ctx_cap) >= 4096;
    L.rows = tc ? (tall ? 256 : 128) : seq_rows <= 16 ? 16 : 64;
    if ((long long)num_tokens * group / L.rows + num_seqs >= (1ll << 31) / num_kv_heads)
        return PKV_ERR_UNSUPPORTED;  // grid
    a.tiles = tile_count(num_tokens, num_seqs, group, L.rows);
    // keys that a tile can see, at most
    long long range = a.ctx_cap;
    if (windowed) {
        const long long w = (long long)window + L.rows / group + 1 + kExtRun;
        if (w < range) range = w;
    }
    if (range < 1) range = 1;
    int parts = 1;
    if (partition_tokens > 0)
        parts = (int)((range + partition_tokens - 1) / partition_tokens);
    else if (partition_tokens == 0)
        parts = auto_parts(num_tokens, num_seqs, num_heads, num_kv_heads, L.rows, pool->head_dim, range);
    a.part_tokens = partition_tokens > 0
                        ? partition_tokens
                        : (int)round_up((size_t)((range + parts - 1) / parts), 128);
    parts = (int)((range + a.part_tokens - 1) / a.part_tokens);
    if ((long long)a.tiles * num_kv_heads * parts >= 1ll << 31) return PKV_ERR_UNSUPPORTED;  // grid
    a.num_parts = parts;
    if (parts > 1) {
        size_t o_bytes;
        const size_t need = partial_bytes((long long)num_tokens * num_heads, pool->head_dim, parts, &o_bytes);
        if (!workspace || workspace_bytes < need) return PKV_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return PKV_ERR_INVALID_ARG;
        a.ws_o = static_cast<float *>(workspace);
        a.ws_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) + o_bytes);
    }
    MapPair maps;
    std::memcpy(&maps, pool->tma, sizeof(maps));
    L.tmk = &maps.k;
    L.tmv = &maps.v;
    const int hd = pool->head_dim;
    const pkv_status st =
        !tc ? launch_extend_fma_f32(L)
        : pool->dtype == PKV_BF16
            ? (hd == 64 ? launch_extend_tc_bf16_d64(L)
                        : (hd == 128 ? launch_extend_tc_bf16_d128(L) : launch_extend_tc_bf16_d256(L)))
            : (hd == 64 ? launch_extend_tc_f16_d64(L)
                        : (hd == 128 ? launch_extend_tc_f16_d128(L) : launch_extend_tc_f16_d256(L)));
    if (st != PKV_OK || parts <= 1) return st;
    return cuda_status(launch_combine(L));
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_extend_workspace_bytes(int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                                  int head_dim, int max_context_len, int partition_tokens) {
    if (num_tokens <= 0 || num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        num_heads % num_kv_heads != 0 || head_dim <= 0 || max_context_len <= 0 || partition_tokens < 0)
        return 0;
    const long long rows = (long long)num_tokens * num_heads;
    size_t o_bytes;
    if (partition_tokens > 0) {
        const long long parts = ((long long)max_context_len + partition_tokens - 1) / partition_tokens;
        return parts <= 1 ? 0 : partial_bytes(rows * parts, head_dim, 1, &o_bytes);
    }
    // The most that any height of tiles takes, in this call or in one of fewer
    // tokens or sequences, which is cut into more parts: wanted items / (tiles *
    // kv heads) parts of at least tokens * group / height tiles.
    long long most = 0;
    for (int height : {16, 64, 128, 256}) {
        const long long parts = most_parts(height, max_context_len);
        if (parts > 1) most = std::max(most, std::min(rows * parts, wanted_items(height, head_dim) * height));
    }
    return most ? partial_bytes(most, head_dim, 1, &o_bytes) : 0;
}

pkv_status pkv_paged_attention_extend(const pkv_pool *pool, void *out, pkv_dtype out_dtype,
                                      const void *query, int num_tokens, int num_seqs,
                                      int num_heads, int num_kv_heads, const int32_t *block_tables,
                                      int max_blocks_per_seq, const int32_t *context_lens,
                                      const int32_t *query_starts, int max_query_len,
                                      int max_context_len, float scale, float softcap, int window,
                                      const float *alibi_slopes, const int32_t *prefix_lens,
                                      int partition_tokens, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    return extend_impl(pool, out, out_dtype, query, num_tokens, num_seqs, num_heads, num_kv_heads,
                       block_tables, max_blocks_per_seq, context_lens, query_starts, max_query_len,
                       max_context_len, scale, softcap, window, alibi_slopes, prefix_lens, false,
                       nullptr, 0, partition_tokens, workspace, workspace_bytes, stream);
}

pkv_status pkv_paged_attention_tree(const pkv_pool *pool, void *out, pkv_dtype out_dtype,
                                    const void *query, int num_tokens, int num_seqs, int num_heads,
                                    int num_kv_heads, const int32_t *block_tables,
                                    int max_blocks_per_seq, const int32_t *context_lens,
                                    const int32_t *query_starts, const uint32_t *tree_mask,
                                    int mask_words, int max_query_len, int max_context_len,
                                    float scale, float softcap, int partition_tokens,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    return extend_impl(pool, out, out_dtype, query, num_tokens, num_seqs, num_heads, num_kv_heads,
                       block_tables, max_blocks_per_seq, context_lens, query_starts, max_query_len,
                       max_context_len, scale, softcap, 0, nullptr, nullptr, true, tree_mask,
                       mask_words, partition_tokens, workspace, workspace_bytes, stream);
}

}  // extern "C"
