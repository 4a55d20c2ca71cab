// tree_decode.cuh - attention of drafted trees over a paged cache.
//
// out[i,h,:] = sum_j p_ij v_j with p = softmax over j of scale * q_i . k_j,
// j running over the cached tokens of node i's sequence and over the nodes of
// its tree whose mask bit is set.
//
// tree_decode_kernel: one warp per (node, query head), a lane holding D/32
// dims, one token at a time with an online softmax in base 2.
#pragma once

#include <cstdint>

#include "decode.cuh"
#include "pagedkv.h"
#include "ptx.cuh"
#include "tree_ops.cuh"

namespace pagedkv {

struct TreeSimpleParams {
    void *out;
    const void *query, *key_cache, *value_cache;
    const int32_t *block_tables, *context_lens, *tree_start, *mask;
    int32_t *dev_err;
    int32_t num_seqs, num_tokens, num_heads, num_kv_heads, num_blocks, block_size;
    int32_t max_blocks_per_seq, mask_words, out_dtype;
    float qk_scale_log2;
};

// The first sequence that row r belongs to, -1 for padding: the lanes of a
// warp look through the offsets.
__device__ __forceinline__ int sequence_of_row(const TreeSimpleParams &p, int limit, int r,
                                               int lane)
{
    for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
        bool mine = false;
        if (s0 + lane < p.num_seqs) {
            const TreeSpan t = tree_span(p.tree_start, s0 + lane, p.num_tokens, limit);
            mine = t.size > 0 && t.first <= r && r - t.first < t.size;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, mine);
        if (hit)
            return s0 + __ffs(hit) - 1;
    }
    return -1;
}

template <typename T, int D> struct TreeRow; // D/32 elements of a cached row per lane
template <int D> struct TreeRow<E4M3, D> {
    static __device__ __forceinline__ void load(const void *cache, int64_t tile, int off, int bs,
                                                int lane, float (&x)[D / 32])
    {
        const uint8_t *t = static_cast<const uint8_t *>(cache) + tile * (bs * D + 4 * bs);
        const float scale = *reinterpret_cast<const float *>(t + bs * D + 4 * off);
        for (int e = 0; e < D / 32; ++e)
            x[e] = static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3 *>(
                       t)[off * D + lane * (D / 32) + e]) * scale;
    }
};
template <typename T, int D> struct TreeRow {
    static __device__ __forceinline__ void load(const void *cache, int64_t tile, int off, int bs,
                                                int lane, float (&x)[D / 32])
    {
        const T *t = static_cast<const T *>(cache) + (tile * bs + off) * D + lane * (D / 32);
        for (int e = 0; e < D / 32; ++e)
            x[e] = static_cast<float>(t[e]);
    }
};

template <typename T, typename QT, int D>
__global__ void __launch_bounds__(128) tree_decode_kernel(
    const __grid_constant__ TreeSimpleParams p)
{
    pdl_launch_dependents();
    pdl_wait_prior_grid();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, h = blockIdx.y * 4 + (threadIdx.x >> 5), r = blockIdx.x;
    if (h >= p.num_heads)
        return;
    const int limit = min(32 * p.mask_words, PA_TREE_MAX_NODES);
    if (r == 0 && h == 0)
        for (int k = lane; k < p.num_seqs; k += 32)
            if (tree_span(p.tree_start, k, p.num_tokens, limit).size < 0)
                report(p.dev_err, PA_DEVERR_TREE);
    const int s = sequence_of_row(p, limit, r, lane);
    if (s < 0)
        return;
    const TreeSpan t = tree_span(p.tree_start, s, p.num_tokens, limit);
    const int bs = p.block_size, ctx = p.context_lens[s];
    const int64_t capacity = min((int64_t)p.max_blocks_per_seq * bs, (int64_t)INT_MAX);
    bool poison = false;
    int n = 0;
    if (ctx < 0 || (int64_t)ctx + t.size > capacity) {
        report(p.dev_err, PA_DEVERR_CONTEXT_LEN);
        poison = true;
    } else {
        n = ctx + t.size;
    }
    float q[E], acc[E];
    const size_t row = ((size_t)r * p.num_heads + h) * D + lane * E;
    for (int e = 0; e < E; ++e) {
        q[e] = static_cast<float>(static_cast<const QT *>(p.query)[row + e]);
        acc[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    bool any = false;
    const int kvh = h / (p.num_heads / p.num_kv_heads);
    const int32_t *words = p.mask + (size_t)r * p.mask_words;
    for (int j = 0; j < n; ++j) {
        const int b = p.block_tables[(size_t)s * p.max_blocks_per_seq + j / bs];
        if (b < 0 || b >= p.num_blocks) {
            report(p.dev_err, PA_DEVERR_BLOCK_ID);
            poison = true;
            continue;
        }
        if (j >= ctx && !((words[(j - ctx) >> 5] >> ((j - ctx) & 31)) & 1))
            continue;
        any = true;
        const int64_t tile = (int64_t)b * p.num_kv_heads + kvh;
        float x[E], dot = 0.f;
        TreeRow<T, D>::load(p.key_cache, tile, j % bs, bs, lane, x);
        for (int e = 0; e < E; ++e)
            dot = fmaf(q[e], x[e], dot);
        for (int o = 16; o > 0; o >>= 1)
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
        dot *= p.qk_scale_log2;
        const float m_new = fmaxf(m, dot);
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        const float keep = exp2f(m - m_use), w = exp2f(dot - m_use);
        TreeRow<T, D>::load(p.value_cache, tile, j % bs, bs, lane, x);
        for (int e = 0; e < E; ++e)
            acc[e] = fmaf(w, x[e], acc[e] * keep);
        l = fmaf(l, keep, w);
        m = m_new;
    }
    for (int e = 0; e < E; ++e)
        store_out(p.out, p.out_dtype, row + e, poison ? NAN : any ? acc[e] / l : 0.f);
}

} // namespace pagedkv
