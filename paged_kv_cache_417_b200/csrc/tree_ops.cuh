// tree_ops.cuh - the index work of a drafted-tree step: ancestor masks, the
// accepted path, and the move of the accepted rows inside the cache.
//
// tree_mask_kernel: ancestors(i) = {i} + ancestors(parent(i)). One CTA per
// tree, one thread per node. Pointer doubling: with up(i) the 2^r-th ancestor
// of i and bits(i) the 2^r nearest nodes of its path, bits(i) |= bits(up(i)),
// up(i) = up(up(i)); a chain of T nodes takes log2(T) rounds instead of T
// steps. Bound by latency (a few dependent loads and barriers; the bytes are
// 4 * (words + 2) a node): B200, one tree of 8 nodes 1.7 us, 256 chains of up
// to 255 nodes 5.3 us (8 rounds of up to 8 words a node; 6.8 us a word at a time).
//
// tree_accept_kernel: one CTA per tree. Every node whose drafted token is
// what the model picked at its parent offers itself as that parent's
// continuation (the lowest index wins, a shared-memory minimum), then one
// thread follows the continuations, at most max_path shared loads. Bound by
// latency: one tree of 8 nodes 1.65 us, 256 of up to 255 nodes 2.1 us.
//
// tree_compact_kernel: row moves along the token axis only, so each
// (cache, head, 16-byte column) is independent of all others: one
// thread owns a column and moves it for every accepted node, in ascending
// order, U loads before their stores. path[k] ascends, so path[k] >= k and a
// store to slot k never hits a row that is still to be read: a later source
// path[k'] > path[k] >= k. No barrier and no staging is needed. Bound by HBM
// for large batches, by its chain of dependent loads (length, path, table
// entry, row) for small ones: 64 sequences, 4 rows each of 2 KB (8 heads x
// 128, f16) in K and V of 32 layers (67 MB read and written, in part in L2)
// 9.1 us, the same of an fp8 cache 8.2 us, one sequence in one layer 2.4 us.
#pragma once

#include <climits>
#include <cstdint>

#include "pagedkv.h"
#include "ptx.cuh"

namespace pagedkv {

struct TreeSpan {
    int32_t first, size; // size < 0: bad offsets
};

// The nodes of sequence s, size -1 when its offsets are bad or it has more
// than `limit` nodes.
__device__ __forceinline__ TreeSpan tree_span(const int32_t *tree_start, int s,
                                              int32_t num_tokens, int32_t limit)
{
    const int32_t a = tree_start[s], b = tree_start[s + 1];
    TreeSpan t;
    t.first = a;
    t.size = b - a;
    if (a < 0 || b < a || b > num_tokens || t.size > limit)
        t.size = -1;
    return t;
}

struct TreeMaskParams {
    int32_t *mask, *depth;
    const int32_t *parents, *tree_start;
    int32_t *dev_err;
    int32_t num_tokens, mask_words;
};

// Threads: 32 * mask_words. Shared memory: threads * (mask_words | 1) words of
// bits (an odd row length spreads the banks),
// then two arrays of `threads` ancestor indices.
__global__ void __launch_bounds__(PA_TREE_MAX_NODES) tree_mask_kernel(
    const __grid_constant__ TreeMaskParams p)
{
    extern __shared__ int32_t tree_smem[];
    pdl_launch_dependents();
    pdl_wait_prior_grid();
    const int W = p.mask_words, stride = W | 1, i = threadIdx.x;
    uint32_t *bits = reinterpret_cast<uint32_t *>(tree_smem);
    int32_t *up = tree_smem + blockDim.x * stride, *up_next = up + blockDim.x;
    const TreeSpan t = tree_span(p.tree_start, blockIdx.x, p.num_tokens, 32 * W);
    if (t.size <= 0) {
        if (t.size < 0 && i == 0)
            report(p.dev_err, PA_DEVERR_TREE);
        return;
    }
    int a = -1;
    if (i < t.size) {
        a = p.parents[t.first + i];
        if (a < -1 || a >= i) {
            report(p.dev_err, PA_DEVERR_TREE);
            a = -1;
        }
        for (int w = 0; w < W; ++w)
            bits[i * stride + w] = w == i >> 5 ? 1u << (i & 31) : 0u;
        up[i] = a;
    }
    // A row is only ever written by its own thread and only gains bits of
    // true ancestors, so it does not matter whether a reader sees its
    // ancestor's row from before or after this round's update: the bits the
    // round needs are in both. The index arrays are double-buffered.
    while (__syncthreads_or(a >= 0)) {
        int a_next = -1;
        if (a >= 0) {
            volatile uint32_t *mine = bits + i * stride, *theirs = bits + a * stride;
            a_next = up[a];
            const int words = (a >> 5) + 1; // the others of that row are zero
            for (int w = 0; w < words; w += 4) {
                uint32_t x[4], y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k] = w + k < words ? theirs[w + k] : 0u;
                    y[k] = w + k < words ? mine[w + k] : 0u;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (w + k < words)
                        mine[w + k] = y[k] | x[k];
            }
        }
        if (i < t.size)
            up_next[i] = a_next;
        a = a_next;
        int32_t *swap = up;
        up = up_next;
        up_next = swap;
    }
    if (p.depth && i < t.size) {
        int n = -1;
        for (int w = 0; w <= i >> 5; ++w)
            n += __popc(bits[i * stride + w]);
        p.depth[t.first + i] = n;
    }
    // blockDim.x = 32 W: every step takes 32 rows further in the same column.
    const int column = i % W;
    for (int r = i / W; r < t.size; r += 32)
        p.mask[(size_t)(t.first + r) * W + column] = (int32_t)bits[r * stride + column];
}

struct TreeAcceptParams {
    int32_t *accepted, *accepted_lens;
    int64_t *next_token;
    const int32_t *parents, *tree_start;
    const int64_t *draft_tokens, *target_tokens;
    int32_t *dev_err;
    int32_t num_tokens, max_path;
};

__global__ void __launch_bounds__(256) tree_accept_kernel(
    const __grid_constant__ TreeAcceptParams p)
{
    __shared__ int32_t follow[PA_TREE_MAX_NODES]; // each node's continuation
    __shared__ int32_t path[PA_TREE_MAX_NODES];
    __shared__ int32_t path_len;
    pdl_launch_dependents();
    pdl_wait_prior_grid();
    const int s = blockIdx.x;
    const TreeSpan t = tree_span(p.tree_start, s, p.num_tokens, PA_TREE_MAX_NODES);
    if (t.size < 0 && threadIdx.x == 0)
        report(p.dev_err, PA_DEVERR_TREE);
    for (int i = threadIdx.x; i < t.size; i += blockDim.x)
        follow[i] = INT_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < t.size; i += blockDim.x) {
        const int a = p.parents[t.first + i];
        if (a < -1 || a >= i)
            report(p.dev_err, PA_DEVERR_TREE);
        else if (a >= 0 && p.draft_tokens[t.first + i] == p.target_tokens[t.first + a])
            atomicMin(&follow[a], i);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int n = 0;
        if (t.size > 0)
            for (int i = 0; i != INT_MAX && n < p.max_path; i = follow[i])
                path[n++] = i;
        path_len = n;
        p.accepted_lens[s] = n;
        p.next_token[s] = n ? p.target_tokens[t.first + path[n - 1]] : -1;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < p.max_path; k += blockDim.x)
        p.accepted[(size_t)s * p.max_path + k] = k < path_len ? path[k] : -1;
}

struct CompactParams {
    void *caches[2 * PA_MAX_LAYERS]; // K and V caches of all layers, each once
    const int32_t *block_tables, *context_lens, *accepted, *accepted_lens;
    int32_t *dev_err;
    int32_t num_blocks, block_size, num_heads, max_blocks_per_seq, max_path;
    int32_t row_vecs;   // 16-byte vectors of a row's elements (or codes)
    int32_t tile_bytes; // of one (block, head) tile
    int32_t scaled;     // fp8: one fp32 scale per row behind the tile's codes
};

// Grid: (sequence, cache).
__global__ void __launch_bounds__(128) tree_compact_kernel(
    const __grid_constant__ CompactParams p)
{
    // Block and row of each accepted node before and after; block -1: not moved.
    __shared__ int32_t src_block[PA_TREE_MAX_NODES], dst_block[PA_TREE_MAX_NODES];
    __shared__ uint8_t src_off[PA_TREE_MAX_NODES], dst_off[PA_TREE_MAX_NODES];
    pdl_launch_dependents();
    pdl_wait_prior_grid();
    const int s = blockIdx.x, tid = threadIdx.x;
    const bool first = blockIdx.y == 0;
    const int n = p.accepted_lens[s], ctx = p.context_lens[s];
    if (n < 0 || n > p.max_path) {
        if (first && tid == 0)
            report(p.dev_err, PA_DEVERR_TREE);
        return;
    }
    const int64_t capacity = min((int64_t)p.max_blocks_per_seq * p.block_size, (int64_t)INT_MAX);
    const int32_t *path = p.accepted + (size_t)s * p.max_path;
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    int bad = 0;
    for (int k = tid; k < n; k += blockDim.x) {
        const int node = path[k];
        if (node < 0 || (k > 0 && node <= path[k - 1])) {
            bad |= PA_DEVERR_TREE;
            continue;
        }
        if (ctx < 0 || (int64_t)ctx + node >= capacity) {
            bad |= PA_DEVERR_CONTEXT_LEN;
            continue;
        }
        const int from = ctx + node, to = ctx + k;
        int sb = table[from / p.block_size], db = table[to / p.block_size];
        if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
            if (first)
                report(p.dev_err, PA_DEVERR_BLOCK_ID);
            sb = db = -1;
        }
        if (node == k)
            sb = db = -1; // in place already
        src_block[k] = sb;
        dst_block[k] = db;
        src_off[k] = (uint8_t)(from % p.block_size);
        dst_off[k] = (uint8_t)(to % p.block_size);
    }
    if (bad && first)
        report(p.dev_err, bad);
    if (__syncthreads_or(bad))
        return;
    char *cache = static_cast<char *>(p.caches[blockIdx.y]);
    const int vecs = p.num_heads * p.row_vecs, columns = vecs + (p.scaled ? p.num_heads : 0);
    const int64_t block_bytes = (int64_t)p.num_heads * p.tile_bytes;
    constexpr int U = 4;
    for (int c = tid; c < columns; c += blockDim.x) {
        const bool scale = c >= vecs;
        const int h = scale ? c - vecs : c / p.row_vecs;
        char *column = cache + (int64_t)h * p.tile_bytes +
                       (scale ? p.block_size * p.row_vecs : c % p.row_vecs) * 16;
        const int row = scale ? 4 : p.row_vecs * 16;
        for (int k0 = 0; k0 < n; k0 += U) {
            uint4 r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u;
                if (k >= n || src_block[k] < 0)
                    continue;
                const char *x = column + src_block[k] * block_bytes + src_off[k] * row;
                if (scale)
                    r[u].x = *reinterpret_cast<const uint32_t *>(x);
                else
                    r[u] = *reinterpret_cast<const uint4 *>(x);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u;
                if (k >= n || src_block[k] < 0)
                    continue;
                char *x = column + dst_block[k] * block_bytes + dst_off[k] * row;
                if (scale)
                    *reinterpret_cast<uint32_t *>(x) = r[u].x;
                else
                    *reinterpret_cast<uint4 *>(x) = r[u];
            }
        }
    }
}

} // namespace pagedkv
