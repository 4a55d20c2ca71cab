// tree.cu - the C ABI's calls for trees of drafted tokens: host-side argument
// checks and kernel launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstring>

#include "pagedkv.h"

#include "host.h"
#include "last_error.h"
#include "tree_decode.cuh"
#include "tree_ops.cuh"

using namespace pagedkv;

namespace {

constexpr int kMaxTreeGroup = 128; // query heads per K/V head

pa_status check_tree_sizes(int32_t num_seqs, int32_t num_tokens)
{
    if (num_seqs < 0 || num_tokens < 0)
        return fail(PA_ERR_INVALID_ARG, "negative size argument");
    if (num_seqs > 65535)
        return fail(PA_ERR_UNSUPPORTED, "num_seqs %d > 65535", num_seqs);
    return PA_OK;
}

pa_status check_mask_words(int32_t mask_words)
{
    if (mask_words < 1 || mask_words > PA_TREE_MAX_NODES / 32)
        return fail(PA_ERR_INVALID_ARG, "mask_words %d outside [1, %d]", mask_words,
                    PA_TREE_MAX_NODES / 32);
    return PA_OK;
}

int tree_ctas() { return kTreeCtasPerSm * sm_count_of_current_device(); }

// Workspace: [records][partial rows][(m, l) pairs], each 256-byte aligned.
struct TreeWorkspace {
    size_t acc, ml, bytes;
};

TreeWorkspace tree_workspace(int ctas, int head_dim)
{
    const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    TreeWorkspace w;
    w.acc = up((size_t)ctas * sizeof(TreeMergeRecord));
    w.ml = w.acc + up((size_t)ctas * 2 * kTreeRows * head_dim * sizeof(float));
    w.bytes = w.ml + up((size_t)ctas * 2 * kTreeRows * sizeof(float2));
    return w;
}

// Rows of a query box: half a tile where that is whole nodes.
int tree_box_rows(int group) { return 64 % group == 0 ? 64 : kTreeRows / group * group; }

// Query rows as (64 elements, heads, nodes, halves of a row): a box holds one
// half of the group's heads of some nodes, rows of 128 bytes in order.
pa_status encode_tree_query(CUtensorMap *map, const void *query, int num_tokens, int num_heads,
                            int group, int head_dim)
{
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc)
        return fail(PA_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
    const cuuint64_t row = (cuuint64_t)head_dim * 2;
    const cuuint64_t dims[4] = {64, (cuuint64_t)num_heads, (cuuint64_t)num_tokens,
                                (cuuint64_t)head_dim / 64};
    const cuuint64_t strides[3] = {row, row * num_heads, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)group, (cuuint32_t)(tree_box_rows(group) / group), 1};
    const cuuint32_t elem_strides[4] = {1, 1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(query), dims,
                           strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return PA_OK;
}

// A 16-bit pool as (64 elements, 8 rows, halves of a row, groups of 8 rows):
// a box is one (block, head) tile, in the layout tree_decode.cuh describes.
pa_status encode_tree_pool(CUtensorMap *map, const void *pool, const pa_cache_desc *c)
{
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc)
        return fail(PA_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
    const cuuint64_t row = (cuuint64_t)c->head_dim * 2;
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)c->head_dim / 64,
                                (cuuint64_t)c->num_blocks * c->num_kv_heads * c->block_size / 8};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)c->head_dim / 64, (cuuint32_t)c->block_size / 8};
    const cuuint32_t elem_strides[4] = {1, 1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(pool), dims,
                           strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return PA_OK;
}

template <typename T, typename QT, int D, int BS>
pa_status launch_tree(const TreeTmaParams &g, int ctas, cudaStream_t st)
{
    using C = TreeCfg<T, D, BS>;
    auto kernel = tree_decode_kernel<T, QT, D, BS>;
    static std::atomic<size_t> smem_set[kMaxDevices];
    cudaError_t e = allow_smem(kernel, C::kSmem, smem_set);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaFuncSetAttribute(tree_decode)");
    e = launch_pdl(kernel, dim3(ctas), dim3(C::kThreads), C::kSmem, st, g);
    if (e != cudaSuccess)
        return cuda_fail(e, "tree_decode launch");
    e = launch_pdl(tree_merge_kernel<D>, dim3(ctas - 1, D / 4 / kMergeCols), dim3(kTreeRows), 0,
                   st, g.p);
    if (e != cudaSuccess)
        return cuda_fail(e, "tree_merge launch");
    return ok();
}

template <typename T, typename QT, int D>
pa_status launch_tree_bs(const TreeTmaParams &g, int block_size, int ctas, cudaStream_t st)
{
    switch (block_size) {
    case 8: return launch_tree<T, QT, D, 8>(g, ctas, st);
    case 16: return launch_tree<T, QT, D, 16>(g, ctas, st);
    case 32: return launch_tree<T, QT, D, 32>(g, ctas, st);
    }
    return fail(PA_ERR_UNSUPPORTED, "block_size %d", block_size);
}

template <typename T, typename QT>
pa_status launch_tree_dim(const TreeTmaParams &g, const pa_cache_desc *c, int ctas,
                          cudaStream_t st)
{
    return c->head_dim == 64 ? launch_tree_bs<T, QT, 64>(g, c->block_size, ctas, st)
                             : launch_tree_bs<T, QT, 128>(g, c->block_size, ctas, st);
}

} // namespace

extern "C" {

pa_status pa_tree_mask(int32_t *mask, int32_t *depth, const int32_t *parents,
                       const int32_t *tree_start, int32_t num_seqs, int32_t num_tokens,
                       int32_t mask_words, int32_t *dev_err, void *stream)
{
    pa_status s = check_tree_sizes(num_seqs, num_tokens);
    if (s != PA_OK)
        return s;
    if ((s = check_mask_words(mask_words)) != PA_OK)
        return s;
    if (num_seqs == 0)
        return ok();
    if (!tree_start || (num_tokens > 0 && (!mask || !parents)))
        return fail(PA_ERR_INVALID_ARG, "NULL pointer argument");
    static std::atomic<size_t> smem_set[kMaxDevices];
    const auto smem_for = [](int words) {
        return (size_t)32 * words * ((words | 1) + 2) * sizeof(int32_t);
    };
    cudaError_t e = allow_smem(tree_mask_kernel, smem_for(PA_TREE_MAX_NODES / 32), smem_set);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaFuncSetAttribute(tree_mask)");
    TreeMaskParams p;
    p.mask = mask;
    p.depth = depth;
    p.parents = parents;
    p.tree_start = tree_start;
    p.dev_err = dev_err;
    p.num_tokens = num_tokens;
    p.mask_words = mask_words;
    e = launch_pdl(tree_mask_kernel, dim3(num_seqs), dim3(32 * mask_words), smem_for(mask_words),
                   static_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess)
        return cuda_fail(e, "tree_mask launch");
    return ok();
}

size_t pa_tree_decode_workspace_size(const pa_cache_desc *cache)
{
    if (check_cache(cache) != PA_OK)
        return (size_t)-1;
    ok();
    return tree_workspace(tree_ctas(), cache->head_dim).bytes;
}

pa_status pa_tree_decode(void *out, pa_dtype out_dtype, const void *query, int32_t num_seqs,
                         int32_t num_tokens, int32_t num_heads, const void *key_cache,
                         const void *value_cache, const pa_cache_desc *cache,
                         const int32_t *block_tables, int32_t max_blocks_per_seq,
                         const int32_t *context_lens, const int32_t *tree_start,
                         const int32_t *mask, int32_t mask_words, float scale, void *workspace,
                         size_t workspace_bytes, int32_t *dev_err, void *stream)
{
    pa_status s = check_cache(cache);
    if (s != PA_OK)
        return s;
    if ((s = check_tree_sizes(num_seqs, num_tokens)) != PA_OK)
        return s;
    if (num_heads <= 0 || max_blocks_per_seq < 0)
        return fail(PA_ERR_INVALID_ARG, "negative size argument");
    if (num_heads % cache->num_kv_heads != 0)
        return fail(PA_ERR_UNSUPPORTED, "num_heads %d is not a multiple of num_kv_heads %d",
                    num_heads, cache->num_kv_heads);
    if (num_heads / cache->num_kv_heads > kMaxTreeGroup)
        return fail(PA_ERR_UNSUPPORTED, "%d query heads per K/V head (at most %d)",
                    num_heads / cache->num_kv_heads, kMaxTreeGroup);
    if (out_dtype != PA_F16 && out_dtype != PA_BF16 && out_dtype != PA_F32)
        return fail(PA_ERR_INVALID_ARG, "out_dtype %d", (int)out_dtype);
    if ((s = check_mask_words(mask_words)) != PA_OK)
        return s;
    if (!(scale == scale))
        return fail(PA_ERR_INVALID_ARG, "scale is NaN");
    if (num_seqs == 0 || num_tokens == 0)
        return ok();
    if (!out || !query || !key_cache || !value_cache || !context_lens || !tree_start || !mask ||
        (max_blocks_per_seq > 0 && !block_tables))
        return fail(PA_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache))
        return fail(PA_ERR_INVALID_ARG, "out, query and caches must be 16-byte aligned");
    if (cache->num_blocks == 0)
        return fail(PA_ERR_INVALID_ARG, "empty pool");
    if ((int64_t)cache->num_blocks * cache->num_kv_heads * (cache->block_size / 8) > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "pool of more than 2^34 rows");
    const size_t need = pa_tree_decode_workspace_size(cache);
    if (!workspace || workspace_bytes < need)
        return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, need);
    if (!aligned16(workspace))
        return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    TreeTmaParams g;
    std::memset(&g, 0, sizeof(g));
    TreeDecodeParams &p = g.p;
    const int ctas = tree_ctas();
    const TreeWorkspace w = tree_workspace(ctas, cache->head_dim);
    char *ws = static_cast<char *>(workspace);
    p.out = out;
    p.key_cache = key_cache;
    p.value_cache = value_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.tree_start = tree_start;
    p.mask = mask;
    p.dev_err = dev_err;
    p.ws_records = reinterpret_cast<TreeMergeRecord *>(ws);
    p.ws_acc = reinterpret_cast<float4 *>(ws + w.acc);
    p.ws_ml = reinterpret_cast<float2 *>(ws + w.ml);
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = cache->num_kv_heads;
    p.group = num_heads / cache->num_kv_heads;
    p.num_blocks = cache->num_blocks;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.mask_words = mask_words;
    p.out_dtype = (int32_t)out_dtype;
    p.q_box_rows = tree_box_rows(p.group);
    // Never zero: a masked score is -infinity times this. The smallest normal
    // number makes every finite score as equal as zero would.
    p.negate = scale < 0.f;
    p.qk_scale_log2 = scale == 0.f ? FLT_MIN : std::fabs(scale) * 1.4426950408889634f;
    if ((s = encode_tree_query(&g.q, query, num_tokens, num_heads, p.group, cache->head_dim)) !=
        PA_OK)
        return s;
    if (cache->dtype == PA_FP8_E4M3)
        return cache->io_dtype == PA_F16 ? launch_tree_dim<E4M3, __half>(g, cache, ctas, st)
                                         : launch_tree_dim<E4M3, __nv_bfloat16>(g, cache, ctas, st);
    if ((s = encode_tree_pool(&g.k, key_cache, cache)) != PA_OK ||
        (s = encode_tree_pool(&g.v, value_cache, cache)) != PA_OK)
        return s;
    return cache->dtype == PA_F16
               ? launch_tree_dim<__half, __half>(g, cache, ctas, st)
               : launch_tree_dim<__nv_bfloat16, __nv_bfloat16>(g, cache, ctas, st);
}

pa_status pa_tree_accept(int32_t *accepted, int32_t *accepted_lens, int64_t *next_token,
                         const int32_t *parents, const int32_t *tree_start,
                         const int64_t *draft_tokens, const int64_t *target_tokens,
                         int32_t num_seqs, int32_t num_tokens, int32_t max_path,
                         int32_t *dev_err, void *stream)
{
    pa_status s = check_tree_sizes(num_seqs, num_tokens);
    if (s != PA_OK)
        return s;
    if (max_path < 1 || max_path > PA_TREE_MAX_NODES)
        return fail(PA_ERR_INVALID_ARG, "max_path %d outside [1, %d]", max_path,
                    PA_TREE_MAX_NODES);
    if (num_seqs == 0)
        return ok();
    if (!accepted || !accepted_lens || !next_token || !tree_start ||
        (num_tokens > 0 && (!parents || !draft_tokens || !target_tokens)))
        return fail(PA_ERR_INVALID_ARG, "NULL pointer argument");
    TreeAcceptParams p;
    p.accepted = accepted;
    p.accepted_lens = accepted_lens;
    p.next_token = next_token;
    p.parents = parents;
    p.tree_start = tree_start;
    p.draft_tokens = draft_tokens;
    p.target_tokens = target_tokens;
    p.dev_err = dev_err;
    p.num_tokens = num_tokens;
    p.max_path = max_path;
    cudaError_t e = launch_pdl(tree_accept_kernel, dim3(num_seqs), dim3(256), 0,
                               static_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess)
        return cuda_fail(e, "tree_accept launch");
    return ok();
}

pa_status pa_tree_compact(void *const *key_caches, void *const *value_caches,
                          int32_t num_layers, const pa_cache_desc *cache,
                          const int32_t *block_tables, int32_t max_blocks_per_seq,
                          const int32_t *context_lens, const int32_t *accepted,
                          const int32_t *accepted_lens, int32_t num_seqs, int32_t max_path,
                          int32_t *dev_err, void *stream)
{
    pa_status s = check_cache(cache);
    if (s != PA_OK)
        return s;
    if ((s = check_tree_sizes(num_seqs, 0)) != PA_OK)
        return s;
    if (num_layers < 1 || num_layers > PA_MAX_LAYERS)
        return fail(PA_ERR_INVALID_ARG, "num_layers %d outside [1, %d]", num_layers, PA_MAX_LAYERS);
    if (max_path < 1 || max_path > PA_TREE_MAX_NODES || max_blocks_per_seq < 0)
        return fail(PA_ERR_INVALID_ARG, "max_path %d (1 .. %d) or max_blocks_per_seq %d", max_path,
                    PA_TREE_MAX_NODES, max_blocks_per_seq);
    if (num_seqs == 0)
        return ok();
    if (!key_caches || !value_caches || !context_lens || !accepted || !accepted_lens ||
        (max_blocks_per_seq > 0 && !block_tables))
        return fail(PA_ERR_INVALID_ARG, "NULL pointer argument");
    CompactParams p;
    std::memset(&p, 0, sizeof(p));
    for (int l = 0; l < num_layers; ++l) {
        if (!key_caches[l] || !value_caches[l])
            return fail(PA_ERR_INVALID_ARG, "NULL cache pointer for layer %d", l);
        if (!aligned16(key_caches[l]) || !aligned16(value_caches[l]))
            return fail(PA_ERR_INVALID_ARG, "cache of layer %d not 16-byte aligned", l);
    }
    // Layers may share a cache, or a layer K and V. Moves in place are not for
    // doing twice (or by two CTAs at once), so each cache is taken once; a
    // table of their addresses, at most half full, finds the repeated ones.
    uint32_t mask = 3;
    while (mask + 1 < 4u * num_layers)
        mask = 2 * mask + 1;
    const void *seen[4 * PA_MAX_LAYERS];
    std::memset(seen, 0, (mask + 1) * sizeof(seen[0]));
    int num_caches = 0;
    for (int i = 0; i < 2 * num_layers; ++i) {
        void *c = i < num_layers ? key_caches[i] : value_caches[i - num_layers];
        uint32_t at = (uint32_t)(reinterpret_cast<uintptr_t>(c) >> 4) * 2654435761u >> 16 & mask;
        while (seen[at] && seen[at] != c)
            at = (at + 1) & mask;
        if (!seen[at]) {
            seen[at] = c;
            p.caches[num_caches++] = c;
        }
    }
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.accepted = accepted;
    p.accepted_lens = accepted_lens;
    p.dev_err = dev_err;
    p.num_blocks = cache->num_blocks;
    p.block_size = cache->block_size;
    p.num_heads = cache->num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_path = max_path;
    p.scaled = cache->dtype == PA_FP8_E4M3;
    p.row_vecs = cache->head_dim * (p.scaled ? 1 : 2) / 16;
    p.tile_bytes = (int32_t)tile_bytes(cache);
    cudaError_t e = launch_pdl(tree_compact_kernel, dim3(num_seqs, num_caches), dim3(128), 0,
                               static_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess)
        return cuda_fail(e, "tree_compact launch");
    return ok();
}

} // extern "C"
