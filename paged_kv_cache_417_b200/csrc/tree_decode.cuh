// tree_decode.cuh - attention of drafted trees over a paged cache.
//
// out[i,h,:] = sum_j p_ij v_j with p = softmax over j of scale * q_i . k_j,
// j running over the cached tokens of node i's sequence and over the nodes of
// its tree whose mask bit is set.
//
// Work. The G query heads of a K/V head and kTreeRows / G consecutive nodes
// make a tile of up to 128 rows that share every key and value: a unit is
// (sequence, K/V head, row tile), its keys cut into tiles of 64 tokens. All
// tiles of all units stand in one line (sequence, head, row tile, tokens
// innermost) that the grid's CTAs, two per SM, cut into equal pieces, whatever
// the lengths: each CTA adds up the lengths itself, so nothing about them is
// needed on the host. A unit cut by the end of a piece leaves partial results
// (m, l, unnormalised rows) in the workspace, at most two per CTA, and
// tree_merge_kernel joins them with the log-sum-exp rule. Row tiles of one
// head follow one another, so their keys come from L2 after the first.
//
// Roles of a CTA's warps:
//   0-3  one thread per row: softmax, and the rescaling and writing of rows
//   4    issues the MMAs: S = Q K^T (128 x 64, both operands in shared
//        memory) and O += P V (128 x D, P in tensor memory)
//   6, 7 fetch Q and K, and V, by TMA, block by block through the block table
//        (one warp for both took 1.5k of the 2.6k cycles of a tile to issue
//        its copies, and held K of the next tile back behind V of this one).
//        They share their schedulers with the softmax warps of the last 64
//        rows, which small trees leave idle; warp 5 is only there to put them
//        where they are.
// Tensor memory (256 columns a CTA): O in D fp32 columns and two S tiles of
// 64; P, 16 bits, overwrites the S tile it comes from. S of the next tile is
// multiplied before P V of this one, so the tensor core works while the
// softmax runs; the other CTA of the SM fills what is left.
//
// Softmax, base 2: p = 2^(s*c - m + kTreeBias), c = scale * log2(e). m is a
// row's reference, not its maximum: it moves (and O and l are rescaled) only
// when a score exceeds it by more than kTreeSlack, which after the first
// tiles of a context is rare. p is then at most 2^(kTreeBias + kTreeSlack),
// inside f16's range, and an f16 p keeps its full precision down to 2^-22 of
// the reference.
//
// Masks. A tile that ends before the context does is seen by every row. Tiles
// at and behind the context's end take the slower path: scores that a row
// does not see become minus infinity. A product
// 0 * NaN would still reach a row, so in those tiles the V rows of nodes and
// behind the last token are looked through, and one that holds a NaN or an
// infinity is zeroed in shared memory and, if it is a node's, added to the
// rows that see it one by one (rescue_rows).
//
// Precision of the weights. P has 16 bits: f16 for f16 rows and fp8 caches, 11
// bits of each weight; bf16 for bf16 rows, 8 bits, where the one-token decode
// multiplies a bf16 head and a bf16 remainder (16 bits). A second product a
// tile would do the same here, for more work on the chain from S to P, which
// bounds larger trees (not measured). Weights' errors are independent, so they add to the rounding
// of a 16-bit output about once more of the same size: against 64 bits the
// error is 1.4 times that of fp32 weights (8 contexts of 16k-32k tokens, bf16:
// 2.3e-3 of the output's size, 1.7e-3; f16: 2.9e-4, 2.1e-4).
//
// Measured (B200), in bursts of 200 calls / in a steady loop, where the power
// limit holds: 96 sequences of 128-2048 tokens, 16 nodes, 32 heads over 8, D
// 128, f16: 91 / 106 us, HBM (5 TB/s in all, 6.1 while the pieces run) and
// uneven ends of the pieces; 33 such sequences, 32 K/V heads: 93 / 111 us; 8
// sequences of 16k-32k tokens, bf16: 152 / 182 us, HBM; 64-node trees: 113 / 137
// us, 706 / 581 TFLOP/s, the chain from S to P of a tile (about 2700 cycles, two
// CTAs overlapping); fp8 with bf16 rows, 64 sequences: 103 / 103 us, the
// widening of codes.
//
// Layouts. K and V blocks lie in shared memory as [8-row group][64-element
// half][8 rows][128 bytes], swizzled, which one 4-D box per block fetches
// whatever the block size. As an operand that is K-major for Q K^T (a row
// group every D / 64 KiB) and MN-major for P V.
#pragma once

#include <climits>
#include <cstdint>
#include <type_traits>

#include <cuda.h>

#include "decode.cuh"
#include "pagedkv.h"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tree_ops.cuh"

namespace pagedkv {

constexpr int kTreeRows = 128;  // rows of a tile: the MMA's M
constexpr int kTreeTile = 64;   // tokens of a tile
constexpr int kTreeCtasPerSm = 2;
constexpr int kSoftmaxWarps = 4, kMmaWarp = 4, kFetchKWarp = 6, kFetchVWarp = 7, kTreeWarps = 8;
constexpr int kRawStages = 2; // fp8 tiles on their way, of K and of V
// Tiles of time that a unit costs beside its own (measured: 3.9 us for a unit
// of one tile, 1.4 us for each further one). us at 2, 4, 6 and 8: 96 sequences
// of 128-2048 tokens, 8 K/V heads, D 128, f16 94.4, 92.6, 93.4, 94.6; fp8 with
// bf16 rows 105.1, 104.0, 105.9, 106.3; 64-node trees 121.5, 116.5, 116.1,
// 116.0; 32 K/V heads 96.2, 94.7, 95.8, 96.2. At D 64 2 is better (f16 69.8,
// 71.5, 73.9, 76.5, fp8 with f16 rows 77.6, 78.6, 80.6, 81.4), by 1-4 %: one
// value for all.
constexpr int kTreeUnitCost = 4;
constexpr float kTreeSlack = 6.f;
constexpr float kTreeBias = 8.f;
// fp8 caches: the least power of two R that V scales are taken relative to.
// p / R is formed in fp32 before a V scale comes in, up to
// 2^(kTreeBias + kTreeSlack) / R, and 64 of them are summed: 2^124. Weights of
// smaller scales lose bits in f16, 2^-25 of R / 2^kTreeBias at most, times a
// code below 2^9: 2^-128 a token, under fp32's normal range. (R / l is normal
// for l up to 2^22, then loses a bit a doubling.)
constexpr float kTreeLeastR = 0x1p-104f;

// Where a unit cut before CTA b's piece (and not earlier) has its parts: part
// 0 in the second slot of the CTA with the piece before, parts 1 .. parts-1
// in the first slots of b and the CTAs with the pieces after.
struct TreeMergeRecord {
    int32_t parts;  // 0: no unit to merge here
    int32_t stride; // of CTAs from one piece to the next
    int32_t rows;
    int32_t first_row; // row of out of the tile's first node
    int32_t kv_head;
};

struct TreeDecodeParams {
    void *out;
    const void *key_cache, *value_cache; // fp8 caches; others come through their maps
    const int32_t *block_tables, *context_lens, *tree_start, *mask;
    int32_t *dev_err;
    TreeMergeRecord *ws_records; // [CTAs]
    float4 *ws_acc;              // [CTAs][2][D / 4][kTreeRows]
    float2 *ws_ml;               // [CTAs][2][kTreeRows] = (m, l)
    int32_t num_seqs, num_tokens, num_heads, num_kv_heads, group, num_blocks;
    int32_t max_blocks_per_seq, mask_words, out_dtype;
    int32_t q_box_rows; // rows of a query box: 64 where the group divides it
    int32_t negate;     // multiply by -Q K^T ...
    float qk_scale_log2; // ... and by this, above zero
};

struct TreeTmaParams {
    CUtensorMap q, k, v;
    TreeDecodeParams p;
};

// A sequence's share of the line of tiles.
struct TreeSeq {
    int32_t first, nodes;  // rows of the packed arrays; nodes 0: nothing to do
    int32_t ctx;
    int32_t row_tiles, tiles; // tiles: of one unit
    int32_t error;            // PA_DEVERR_* bits
    bool bad_context;         // rows become NaN (one tile per unit, nothing read)
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeDecodeParams &p, int s, int bs)
{
    TreeSeq q;
    const TreeSpan t =
        tree_span(p.tree_start, s, p.num_tokens, min(32 * p.mask_words, PA_TREE_MAX_NODES));
    q.first = t.first;
    q.nodes = max(t.size, 0);
    q.error = t.size < 0 ? PA_DEVERR_TREE : 0;
    q.ctx = p.context_lens[s];
    // Below 2^31 by two tiles, so that no sum of positions overflows.
    const int64_t capacity =
        min((int64_t)p.max_blocks_per_seq * bs, (int64_t)INT_MAX - 2 * kTreeTile);
    q.bad_context = q.nodes > 0 && (q.ctx < 0 || (int64_t)q.ctx + q.nodes > capacity);
    if (q.bad_context)
        q.error |= PA_DEVERR_CONTEXT_LEN;
    const int per_tile = kTreeRows / p.group;
    q.row_tiles = (q.nodes + per_tile - 1) / per_tile;
    q.tiles = q.nodes == 0       ? 0
              : q.bad_context ? 1
                              : (int)(((int64_t)q.ctx + q.nodes + kTreeTile - 1) / kTreeTile);
    return q;
}

__device__ __forceinline__ int64_t tree_seq_places(const TreeDecodeParams &p, const TreeSeq &q)
{
    return (int64_t)(q.tiles + kTreeUnitCost) * q.row_tiles * p.num_kv_heads;
}

// What a CTA does. The line has kTreeUnitCost + tiles places per unit, and of
// n = `pieces` pieces piece b begins at place b * total / n: the first
// kTreeUnitCost places of a unit stand for its fixed cost (query rows, the
// masked tiles at its end, the epilogue), so that a piece of many short units
// takes as long as one of a few long ones. A piece that begins in them begins
// with the unit's first tile.
struct TreePlan {
    int64_t begin, end;      // places of the line
    int32_t stride, lane;    // CTAs that share a piece, and which of them this is
    int64_t each;            // total / pieces
    int32_t pieces, rest;    // rest: total % pieces
    int64_t unit_begin;      // first place of the unit that `begin` is in
    int32_t seq, unit, tile; // that unit of the sequence, and the piece's first tile of it
    bool empty;              // no tile in this piece
    TreeSeq q;               // that sequence

    __device__ __forceinline__ int64_t piece(int b) const
    {
        return b * each + (uint32_t)(b * rest) / (uint32_t)pieces;
    }
    // The end of this piece among the tiles of a unit.
    __device__ __forceinline__ int tile_end(int64_t first_place, int tiles) const
    {
        return (int)max((int64_t)0, min((int64_t)tiles, end - first_place - kTreeUnitCost));
    }
    // The thread whose sequence q, beginning at `first`, holds `begin`.
    __device__ __forceinline__ void locate(const TreeSeq &at, int s, int64_t first)
    {
        q = at;
        const int places = q.tiles + kTreeUnitCost;
        seq = s;
        unit = (int)((begin - first) / places);
        unit_begin = first + (int64_t)unit * places;
        tile = max(0, (int)(begin - unit_begin) - kTreeUnitCost);
        empty = tile_end(unit_begin, q.tiles) <= tile;
    }
};

// Adds up the tiles of all sequences, every thread of the CTA taking part;
// `plan` and `sums` (32 entries) are in shared memory. Ends with a barrier.
__device__ __forceinline__ void tree_plan(const TreeDecodeParams &p, int bs, TreePlan *plan,
                                          int64_t *sums)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nwarps = blockDim.x >> 5;
    const bool one = p.num_seqs <= (int)blockDim.x; // the usual case: one sequence per thread
    int64_t total = 0, mine = 0, before = 0;
    int32_t error = 0, odd = 0;
    TreeSeq q;
    for (int s0 = 0; s0 < p.num_seqs; s0 += blockDim.x) {
        const int s = s0 + tid;
        if (s < p.num_seqs) {
            q = tree_seq(p, s, bs);
            error |= q.error;
            odd |= q.row_tiles & 1;
            mine = tree_seq_places(p, q);
            total += mine;
        }
    }
    if (error && blockIdx.x == 0)
        report(p.dev_err, error);
    // Where every tree has an even number of row tiles, two CTAs share each
    // piece, one for the even and one for the odd ones: both then read the
    // same keys and values at the same time, and L2 once.
    const int halve = __syncthreads_or(odd) ? 0 : 1, stride = 1 + halve;
    mine >>= halve;
    total >>= halve;
    int64_t upto = one ? mine : total; // inclusive sums over threads
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o)
            upto += x;
    }
    if (lane == 31)
        sums[warp] = upto;
    __syncthreads();
    total = 0;
    for (int w = 0; w < nwarps; ++w) {
        if (w == warp)
            before = total;
        total += sums[w];
    }
    const int pieces = (int)min((int64_t)(gridDim.x >> halve), total);
    const int piece = blockIdx.x >> halve;
    if (tid == 0) {
        plan->pieces = pieces;
        plan->stride = stride;
        plan->lane = blockIdx.x & halve;
        plan->empty = true;
        if (piece < pieces) {
            plan->each = total / pieces;
            plan->rest = (int)(total % pieces);
            plan->begin = plan->piece(piece);
            plan->end = plan->piece(piece + 1);
        }
    }
    __syncthreads();
    if (piece >= pieces)
        return;
    const int64_t begin = plan->begin;
    if (one) {
        const int64_t first = before + upto - mine;
        if (mine > 0 && first <= begin && begin < first + mine) {
            plan->locate(q, tid, first);
        }
        __syncthreads();
        return;
    }
    // More sequences than threads: again, in order, until the piece is found.
    int64_t base = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += blockDim.x) {
        mine = 0;
        if (s0 + tid < p.num_seqs) {
            q = tree_seq(p, s0 + tid, bs);
            mine = tree_seq_places(p, q) >> halve;
        }
        upto = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o)
                upto += x;
        }
        __syncthreads();
        if (lane == 31)
            sums[warp] = upto;
        __syncthreads();
        int64_t chunk = 0;
        for (int w = 0; w < nwarps; ++w) {
            if (w == warp)
                before = chunk;
            chunk += sums[w];
        }
        const int64_t first = base + before + upto - mine;
        if (mine > 0 && first <= begin && begin < first + mine) {
            plan->locate(q, s0 + tid, first);
        }
        base += chunk;
        if (base > begin)
            break; // the same for every thread
    }
    __syncthreads();
}

// One unit's share of a CTA's piece, as the fetching warp hands it on.
struct TreeSegment {
    int32_t tile0, tile1; // tokens [64 * tile0, 64 * tile1)
    int32_t ctx, n;       // cached tokens, and with the tree
    int32_t row0;         // packed row of the tile's first node
    int32_t rows;         // live rows of the tile
    int32_t kv_head;
    int32_t slot;         // -1: writes its rows; 0, 1: leaves a part in that slot
    int32_t q_at;         // byte offset of its query rows in the query area
    int32_t last;         // 1: the CTA's last segment
};

template <typename T, int D, int BS> struct TreeCfg {
    static constexpr bool kFp8 = std::is_same<T, E4M3>::value;
    // The type of P V: e4m3 codes and weights go into f16 better than into
    // bf16; K takes the query rows' type.
    using PT = std::conditional_t<kFp8, __half, T>;
    static constexpr int kHalves = D / 64;
    static constexpr int kTileBytes = kTreeTile * D * 2;       // a K or V tile
    static constexpr int kQBytes = kTreeRows * D * 2;
    static constexpr int kGroupBytes = 1024 * kHalves;         // 8 rows
    static constexpr int kStages = (D == 128 ? 2 : 4) / (kFp8 ? 2 : 1); // of K and of V
    static constexpr int kBlocks = kTreeTile / BS;             // blocks of a tile
    // Bytes of a block in memory, and of the ring that fp8 tiles arrive in.
    static constexpr int kBlockBytes = kFp8 ? BS * D + 4 * BS : BS * D * 2;
    static constexpr int kRawBytes = kFp8 ? kBlocks * kBlockBytes : 0;
    static constexpr int kThreads = 32 * kTreeWarps;
    static constexpr int kSmem =
        1024 + kQBytes + 2 * kStages * kTileBytes + 2 * kRawStages * kRawBytes;
    static constexpr uint32_t kColumns = 256;
    static constexpr uint32_t kS0 = D; // tensor-memory column of the first S tile
};

// Barriers and small state of a CTA.
template <int NS> struct TreeShared {
    uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
    // By segment; q_empty by its parity.
    uint64_t d_full[4], q_full[4], q_empty[2], s_full[2], p_full[2], o_full, o_free, warps, drain;
    TreePlan plan;
    int64_t sums[32];
    TreeSegment seg[4];
    int32_t poison[4];       // segment met a block id outside the pool
    // Tokens of a tile whose V row holds NaN or infinity, by the tile's parity:
    // a warp that sets bits for tile it + 2 has met all others after tile it + 1
    // set its own (sync_warps), which is after each of them has read tile it's.
    // One buffer would let a warp with nothing else to do in a tile set the
    // next one's bits before a late warp has read this one's.
    uint32_t strange[2][2];
    // fp8 caches: raw tiles, and the row scales of four tiles.
    uint64_t raw_full[2][kRawStages], ks_full[4], vs_full[4];
    alignas(16) float ks[4][kTreeTile]; // times scale * log2(e)
    alignas(16) float vs[4][kTreeTile];
    float vmax[4]; // the largest finite V scale in size of a tile that every row sees
    uint32_t tmem;
    int32_t keep_o;          // tile whose P V adds to O although it is a segment's first
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats to a packed pair, the first in the low half.
template <typename QT> __device__ __forceinline__ uint32_t pack2(float a, float b)
{
    uint32_t r;
    if constexpr (std::is_same<QT, __half>::value)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Byte address inside a K or V tile of 16-byte piece c (of D / 8) of row j.
template <int D> __device__ __forceinline__ uint32_t tree_piece_at(int j, int c)
{
    return (j >> 3) * (1024 * (D / 64)) + (c >> 3) * 1024 + (j & 7) * 128 +
           (((c & 7) ^ (j & 7)) << 4);
}

// Which of the 64 tokens of a tile a row sees: those before the context's
// end, then those whose bit is set in its mask row. The words are loaded
// ahead of their use.
struct TreeSeen {
    uint32_t w[3];
    __device__ __forceinline__ void load(const int32_t *words, int num_words, int t0, int ctx)
    {
        const int first = max(t0 - ctx, 0) >> 5;
#pragma unroll
        for (int k = 0; k < 3; ++k)
            w[k] = first + k < num_words ? (uint32_t)words[first + k] : 0u;
    }
    __device__ __forceinline__ uint64_t bits(int t0, int ctx, int n) const
    {
        const int b0 = t0 - ctx; // node of column 0; negative: cached tokens first
        uint64_t b = ~0ull;
        if (b0 >= 0)
            b = (uint64_t)__funnelshift_r(w[0], w[1], b0) |
                ((uint64_t)__funnelshift_r(w[1], w[2], b0) << 32);
        else if (b0 > -kTreeTile)
            b = (((uint64_t)w[1] << 32 | w[0]) << -b0) | ((1ull << -b0) - 1);
        if (n - t0 < kTreeTile)
            b &= n > t0 ? (1ull << (n - t0)) - 1 : 0ull;
        return b;
    }
};

// 32 bytes to 32-byte (wide) or 16-byte aligned memory.
__device__ __forceinline__ void store32(void *to, const uint32_t *w, bool wide)
{
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                     "r"(w[7])
                     : "memory");
    else {
        static_cast<uint4 *>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// 32 (4) consecutive floats of a row to `out`, rounded to its type. A thread
// per row makes every store of a warp touch 32 lines, so each takes a whole
// sector where `out` is aligned to one.
__device__ __forceinline__ void store_row32(void *out, int dtype, size_t at, const uint32_t (&o)[32])
{
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    if (dtype == 2) {
#pragma unroll
        for (int k = 0; k < 32; k += 8)
            store32(static_cast<float *>(out) + at + k, o + k, wide);
        return;
    }
    uint32_t w[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float a = __uint_as_float(o[2 * k]), b = __uint_as_float(o[2 * k + 1]);
        w[k] = dtype == 0 ? pack2<__half>(a, b) : pack2<__nv_bfloat16>(a, b);
    }
#pragma unroll
    for (int k = 0; k < 16; k += 8)
        store32(static_cast<uint16_t *>(out) + at + 2 * k, w + k, wide);
}

__device__ __forceinline__ void store_row4(void *out, int dtype, size_t at, float4 v)
{
    if (dtype == 2) {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = v;
        return;
    }
    uint2 w;
    w.x = dtype == 0 ? pack2<__half>(v.x, v.y) : pack2<__nv_bfloat16>(v.x, v.y);
    w.y = dtype == 0 ? pack2<__half>(v.z, v.w) : pack2<__nv_bfloat16>(v.z, v.w);
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) = w;
}

// O += p * v for the `strange` tokens of a V tile, each for the rows that see
// it; every softmax thread with its own row. `p_column` is the first column
// of this tile's P in the warp's lanes, `o_column` of O.
template <typename QT, int D>
__device__ __noinline__ void rescue_rows(uint64_t strange, uint64_t seen, uint32_t v_tile,
                                         uint32_t p_column, uint32_t o_column)
{
    for (; strange; strange &= strange - 1) {
        const int j = __ffsll((long long)strange) - 1;
        const uint32_t pair = tmem_ld_x1(p_column + (j >> 1));
        const float2 both = Elem<QT>::pair(pair);
        const float pj = j & 1 ? both.y : both.x;
        const bool mine = (seen >> j) & 1;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tmem_ld_x32(o_column + c0, o);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint4 raw;
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w)
                             : "r"(v_tile + tree_piece_at<D>(j, c0 / 8 + c)));
                float v[8];
                unpack8_to<QT>(raw, v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (mine)
                        o[8 * c + e] = __float_as_uint(
                            fmaf(pj, v[e], __uint_as_float(o[8 * c + e])));
            }
            tmem_st_x32(o_column + c0, o);
        }
        tmem_wait_st();
    }
}

// Whether a 16-byte piece of 16-bit elements holds a NaN or an infinity.
template <typename QT> __device__ __forceinline__ bool not_finite(const uint4 &x)
{
    constexpr uint32_t E = std::is_same<QT, __half>::value ? 0x7c00u : 0x7f80u;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        bad |= (w[k] & E) == E || ((w[k] >> 16) & E) == E;
    return bad;
}

// The fetching warps: K tiles of the CTA's piece, with each segment's
// description and query rows, or its V tiles. One body for both: the roles of
// this kernel run at once and share the instruction cache.
//
// fp8 tiles come as they are (codes and row scales, one bulk copy per block)
// into a ring of kRawStages, and are widened from there to the swizzled
// 16-bit tile by the same warp while the next one is on its way. Scores are
// multiplied by K's scales and weights by V's in the softmax; the scales go
// to it on their own barriers.
template <typename T, typename QT, int D, int BS>
__device__ __forceinline__ void tree_fetch(const TreeTmaParams &g, const bool is_v,
                                           TreeShared<TreeCfg<T, D, BS>::kStages> &sh,
                                           uint32_t q_tile, uint32_t ring, uint32_t raw_ring,
                                           bool &ok)
{
    using C = TreeCfg<T, D, BS>;
    constexpr int NS = C::kStages;
    const TreeDecodeParams &p = g.p;
    const int lane = threadIdx.x & 31, per_tile = kTreeRows / p.group;
    const auto wait = [&](uint64_t &bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu,
                        ok && mbar_wait_suspended(smem_addr(&bar), parity, kWaitLimitNs));
        return ok;
    };
    uint64_t *full = is_v ? sh.v_full : sh.k_full, *empty = is_v ? sh.v_empty : sh.k_empty;
    const CUtensorMap *map = is_v ? &g.v : &g.k;
    const uint8_t *pool = static_cast<const uint8_t *>(is_v ? p.value_cache : p.key_cache);
    int s = sh.plan.seq;
    TreeSeq q = sh.plan.q;
    const int stride = sh.plan.stride;
    // Keys and values that are read once leave L2 to the partial results and
    // query rows (33 sequences of 32 K/V heads 97 -> 94 us, the 8-head layer 94
    // -> 92); those of several row tiles stay for the tiles that follow (three
    // tiles over 4 contexts of 32k, bf16: 273 -> 264 us; trees of one and two
    // over 256-4096 tokens 112.0 -> 109.5).
    uint64_t policy = l2_policy(q.row_tiles == 1);
    int64_t unit_begin = sh.plan.unit_begin;
    int unit = sh.plan.unit, tile = sh.plan.tile, it = 0, seg = 0;
    // Widens tile `of` of the CTA, the first `blocks` blocks of which came.
    const auto widen = [&](int of, int blocks, int left) {
        if constexpr (C::kFp8) {
            const int st = of % NS, raw_st = of % kRawStages;
            if (!wait(sh.raw_full[is_v][raw_st], (of / kRawStages) & 1))
                return;
            const uint32_t raw = raw_ring + raw_st * C::kRawBytes;
            float *scales = is_v ? sh.vs[of & 3] : sh.ks[of & 3];
            // Rows of V whose scale is no finite number come in full (inf and
            // NaN are 16-bit values too) with a scale of one, rows behind the
            // last token with zero: weights of zero then stay zero.
            uint32_t odd[2] = {0, 0};
            const auto publish = [&]() {
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int j = lane + 32 * k;
                    float x;
                    asm volatile("ld.shared.f32 %0, [%1];"
                                 : "=f"(x)
                                 : "r"(raw + (j / BS) * C::kBlockBytes + BS * D + (j % BS) * 4)
                                 : "memory");
                    if (is_v) {
                        x = j < left ? x : 0.f;
                        const bool fine = fabsf(x) < INFINITY;
                        odd[k] = __ballot_sync(0xffffffffu, !fine);
                        top = fine ? fmaxf(top, fabsf(x)) : top;
                        scales[j] = fine ? x : 1.f;
                    } else {
                        scales[j] = x * p.qk_scale_log2;
                    }
                }
                if (is_v) {
                    for (int o = 16; o > 0; o >>= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    if (lane == 0)
                        sh.vmax[of & 3] = top;
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(is_v ? &sh.vs_full[of & 3] : &sh.ks_full[of & 3]));
            };
            // V's scales are wanted before its tile is free; K's with it.
            if (is_v)
                publish();
            if (of >= NS && !wait(empty[st], ((of / NS) & 1) ^ 1))
                return;
            if (!is_v)
                publish();
            // A step takes 32 chunks of 16 codes: kRows rows, a chunk a lane.
            constexpr int kChunks = D / 16, kRows = 32 / kChunks;
            const int i = lane % kChunks, r0 = lane / kChunks;
            // Lanes of a row's second half store their two pieces in the
            // other order: 8 lanes then meet 8 different bank groups.
            const bool turn = i >= 4;
            uint32_t at[8 / kRows][2]; // in a group of 8 rows, for each of its steps
#pragma unroll
            for (int q = 0; q < 8 / kRows; ++q)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    at[q][u] = ring + st * C::kTileBytes +
                               tree_piece_at<D>(q * kRows + r0, 2 * i + (turn ? 1 - u : u));
            const bool bf16 = !is_v && std::is_same<QT, __nv_bfloat16>::value;
#pragma unroll 1
            for (int b = 0; b < blocks; ++b) {
                const uint32_t from = raw + b * C::kBlockBytes + lane * 16;
                // All of a block's loads before its stores, for their latency.
                uint4 codes[BS / kRows];
#pragma unroll
                for (int r = 0; r < BS; r += kRows) {
                    uint4 &code = codes[r / kRows];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(code.x), "=r"(code.y), "=r"(code.z), "=r"(code.w)
                                 : "r"(from + r * D)
                                 : "memory");
                }
#pragma unroll
                for (int r = 0; r < BS; r += kRows) {
                    const uint4 code = codes[r / kRows];
                    uint32_t w[8];
                    Store<E4M3>::to_h2(turn ? make_uint4(code.z, code.w, code.x, code.y) : code,
                                       w);
                    if (bf16) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 f = h2_to_float2(w[e]);
                            w[e] = pack2<__nv_bfloat16>(f.x, f.y);
                        }
                    }
                    const uint32_t group = (b * BS + r) / 8 * C::kGroupBytes;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         at[r % 8 / kRows][u] + group),
                                     "r"(w[4 * u]), "r"(w[4 * u + 1]), "r"(w[4 * u + 2]),
                                     "r"(w[4 * u + 3])
                                     : "memory");
                }
            }
            for (uint64_t rows = (uint64_t)odd[1] << 32 | odd[0]; rows; rows &= rows - 1) {
                const int j = __ffsll((long long)rows) - 1;
                const uint32_t tile_of = raw + (j / BS) * C::kBlockBytes;
                __syncwarp();
                for (int e = lane; e < D; e += 32) {
                    uint32_t code;
                    float scale;
                    asm volatile("ld.shared.u8 %0, [%1];"
                                 : "=r"(code)
                                 : "r"(tile_of + (j % BS) * D + e)
                                 : "memory");
                    asm volatile("ld.shared.f32 %0, [%1];"
                                 : "=f"(scale)
                                 : "r"(tile_of + BS * D + (j % BS) * 4)
                                 : "memory");
                    float f[4];
                    e4m3x4_to_float(code, f);
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(ring + st * C::kTileBytes +
                                                                 tree_piece_at<D>(j, e / 8) +
                                                                 e % 8 * 2),
                                 "h"((uint16_t)pack2<typename C::PT>(f[0] * scale, 0.f))
                                 : "memory");
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&full[st]));
        }
    };
    int to_widen = 0, to_widen_left = 0; // blocks and tokens of the tile before
    uint32_t q_seen[2] = {0, 0}; // segments of each parity whose query rows were seen done
    bool was_whole = false;
    int issued = 0, segs_issued = 0; // tiles and query rows whose copies were issued
    for (bool last = false; !last && ok; ++seg) {
        const int row_tiles = q.row_tiles >> (stride - 1); // this CTA's
        const int rt = unit % row_tiles * stride + sh.plan.lane, h = unit / row_tiles;
        const int tile0 = tile, end = sh.plan.tile_end(unit_begin, q.tiles);
        unit_begin += q.tiles + kTreeUnitCost;
        last = sh.plan.end <= unit_begin + kTreeUnitCost; // no tile of the next unit
        const int n = q.bad_context ? 0 : q.ctx + q.nodes;
        const int32_t *table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
        const auto block_id = [&](int t) { // lane's block of tile t, -1: none
            const int b = t * C::kBlocks + lane;
            return lane < C::kBlocks && b * BS < n ? table[b] : -1;
        };
        int id = block_id(tile);
        for (; tile < end; ++tile, ++it) {
            const int st = it % NS;
            const uint32_t ph = (it / NS) & 1;
            const int left = n - tile * kTreeTile; // tokens from here on
            const int blocks = left <= 0 ? 0 : min(C::kBlocks, (left + BS - 1) / BS);
            const int next = tile + 1 < end ? block_id(tile + 1) : -1;
            if (!C::kFp8 && it >= NS && !wait(empty[st], ph ^ 1))
                break;
            // Only now, so that the table's latency passes during the wait.
            const bool bad = lane < blocks && (id < 0 || id >= p.num_blocks);
            const bool any_bad = __any_sync(0xffffffffu, bad);
            const int tile_at = (bad ? 0 : id) * p.num_kv_heads + h; // (block, head) tile
            const uint32_t bar = smem_addr(C::kFp8 ? &sh.raw_full[is_v][it % kRawStages]
                                                   : &full[st]);
            const uint32_t to = C::kFp8 ? raw_ring + (it % kRawStages) * C::kRawBytes
                                        : ring + st * C::kTileBytes;
            int from[C::kBlocks];
#pragma unroll
            for (int b = 0; b < C::kBlocks; ++b)
                from[b] = __shfl_sync(0xffffffffu, tile_at, b);
            if (elect_one()) {
                if (is_v && tile == tile0)
                    sh.poison[seg & 3] = q.bad_context;
                if (any_bad) {
                    report(p.dev_err, PA_DEVERR_BLOCK_ID);
                    if (is_v)
                        sh.poison[seg & 3] = 1;
                }
                mbar_arrive_expect_tx(bar, blocks * C::kBlockBytes);
#pragma unroll
                for (int b = 0; b < C::kBlocks; ++b) {
                    if (b >= blocks)
                        break;
                    if constexpr (C::kFp8)
                        bulk_g2s(to + b * C::kBlockBytes,
                                 pool + (int64_t)from[b] * C::kBlockBytes, C::kBlockBytes, bar);
                    else
                        tma_load_4d(to + b * C::kBlockBytes, map, 0, 0, 0, from[b] * (BS / 8),
                                    bar, policy);
                }
            }
            __syncwarp();
            issued = it + 1;
            if constexpr (C::kFp8) {
                if (it > 0)
                    widen(it - 1, to_widen, to_widen_left);
                if (!ok)
                    break;
                to_widen = blocks;
                to_widen_left = left;
            }
            if (!is_v && tile == tile0) {
                // A segment of up to 64 rows takes half of the query area,
                // so that its rows can come while the last segment's are
                // still multiplied; a larger one takes all of it.
                const int rows = min(per_tile, q.nodes - rt * per_tile) * p.group;
                const bool whole = rows > 64 || p.q_box_rows != 64;
                const auto q_free = [&](int of) { // segment `of`'s rows are done with
                    if (of >= 0 && (q_seen[of & 1] <= of >> 1))
                        return wait(sh.q_empty[of & 1], q_seen[of & 1]++ & 1);
                    return true;
                };
                if (!q_free(seg - 2) || ((whole || was_whole) && !q_free(seg - 1)))
                    break;
                was_whole = whole;
                if (elect_one()) {
                    TreeSegment d;
                    d.tile0 = tile0;
                    d.tile1 = end;
                    d.ctx = q.bad_context ? 0 : q.ctx;
                    d.n = n;
                    d.row0 = q.first + rt * per_tile;
                    d.rows = rows;
                    d.kv_head = h;
                    d.slot = tile0 > 0 ? 0 : end < q.tiles ? 1 : -1;
                    d.q_at = whole ? 0 : (seg & 1) * 8192;
                    d.last = last;
                    sh.seg[seg & 3] = d;
                    mbar_arrive(smem_addr(&sh.d_full[seg & 3]));
                    const uint32_t qbar = smem_addr(&sh.q_full[seg & 3]);
                    const int boxes = p.q_box_rows == 64 && rows > 64 ? 2 : 1;
                    mbar_arrive_expect_tx(qbar, boxes * p.q_box_rows * 128 * C::kHalves);
                    for (int b = 0; b < boxes; ++b)
                        for (int u = 0; u < C::kHalves; ++u)
                            tma_load_4d(q_tile + d.q_at + u * (kTreeRows * 128) + b * 8192, &g.q,
                                        0, h * p.group, d.row0 + b * (64 / p.group), u, qbar);
                }
                __syncwarp();
                segs_issued = seg + 1;
            }
            id = next;
        }
        if (!ok)
            break;
        // The next unit: of this sequence, or of the next one with any.
        tile = 0;
        if (++unit == row_tiles * p.num_kv_heads && !last) {
            unit = 0;
            for (++s; s < p.num_seqs; s += 32) {
                const bool has = s + lane < p.num_seqs && tree_seq(p, s + lane, BS).nodes > 0;
                const unsigned hit = __ballot_sync(0xffffffffu, has);
                if (hit) {
                    s += __ffs(hit) - 1;
                    break;
                }
            }
            if (s >= p.num_seqs) { // the lengths changed under this call: stop, in bounds
                ok = false;
                break;
            }
            q = tree_seq(p, s, BS);
            policy = l2_policy(q.row_tiles == 1);
        }
    }
    if (C::kFp8 && ok)
        widen(it - 1, to_widen, to_widen_left);
    if (!ok) {
        // Let the copies in flight land before the CTA goes: those of the last
        // kRing tiles issued, and of the last two segments' query rows (older
        // ones were waited for before theirs could be overwritten). Waiting for
        // a phase that was not begun would return at once with the one before
        // it still open, so only what was issued counts.
        constexpr uint64_t kDrainNs = 10000000;
        constexpr int kRing = C::kFp8 ? kRawStages : NS;
        for (int i = max(0, issued - kRing); i < issued; ++i)
            mbar_wait_bounded(smem_addr(C::kFp8 ? &sh.raw_full[is_v][i % kRing] : &full[i % kRing]),
                              (i / kRing) & 1, kDrainNs);
        for (int i = max(0, segs_issued - 2); i < segs_issued; ++i)
            mbar_wait_bounded(smem_addr(&sh.q_full[i & 3]), (i >> 2) & 1, kDrainNs);
    }
}

// T: the cache's storage, QT: the type of query rows and of the products.
template <typename T, typename QT, int D, int BS>
__global__ void __launch_bounds__(TreeCfg<T, D, BS>::kThreads, kTreeCtasPerSm)
    tree_decode_kernel(const __grid_constant__ TreeTmaParams g)
{
    using C = TreeCfg<T, D, BS>;
    constexpr int NS = C::kStages;
    constexpr bool kBf16 = std::is_same<QT, __nv_bfloat16>::value;
    using PT = typename C::PT;
    extern __shared__ __align__(1024) uint8_t tree_dyn[];
    __shared__ TreeShared<NS> sh;
    const TreeDecodeParams &p = g.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(tree_dyn) + 1023u) & ~1023u;
    const uint32_t q_tile = base, k_tiles = base + C::kQBytes,
                   v_tiles = k_tiles + NS * C::kTileBytes,
                   raw_tiles = v_tiles + NS * C::kTileBytes;

    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_addr(&sh.k_full[i]), 1);
            mbar_init(smem_addr(&sh.k_empty[i]), 1);
            mbar_init(smem_addr(&sh.v_full[i]), 1);
            mbar_init(smem_addr(&sh.v_empty[i]), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_addr(&sh.d_full[i]), 1);
            mbar_init(smem_addr(&sh.ks_full[i]), 1);
            mbar_init(smem_addr(&sh.vs_full[i]), 1);
            mbar_init(smem_addr(&sh.q_full[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.q_empty[i]), 1);
            for (int k = 0; k < kRawStages; ++k)
                mbar_init(smem_addr(&sh.raw_full[i][k]), 1);
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.p_full[i]), kSoftmaxWarps);
        }
        mbar_init(smem_addr(&sh.o_full), 1);
        mbar_init(smem_addr(&sh.o_free), kSoftmaxWarps);
        mbar_init(smem_addr(&sh.warps), kSoftmaxWarps);
        mbar_init(smem_addr(&sh.drain), 1);
        fence_mbar_init();
        sh.keep_o = -1;
        sh.strange[0][0] = sh.strange[0][1] = sh.strange[1][0] = sh.strange[1][1] = 0;
    }
    if (warp == kMmaWarp)
        tmem_alloc(smem_addr(&sh.tmem), C::kColumns);
    tcgen05_fence_before();
    pdl_wait_prior_grid();
    tree_plan(p, BS, &sh.plan, sh.sums);
    tcgen05_fence_after();
    const uint32_t tmem = sh.tmem;
    bool ok = true;
    // Parts that this CTA does not come to write (a wait that runs out, lengths
    // that change under the call) must not be merged from what a call before
    // left there: l = NaN makes rows of them NaN. The thread that fills a row
    // later is the one that stores here.
    if (tid < kTreeRows) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            __stcg(p.ws_ml + ((size_t)blockIdx.x * 2 + k) * kTreeRows + tid,
                   make_float2(-INFINITY, NAN));
    }
    const auto wait = [&](uint64_t &bar, uint32_t parity) {
        ok = ok && mbar_wait_suspended(smem_addr(&bar), parity, kWaitLimitNs);
        return ok;
    };

    if (sh.plan.empty) {
        if (tid == 0)
            p.ws_records[blockIdx.x].parts = 0;
    } else if (warp == kFetchKWarp || warp == kFetchVWarp) {
        const bool is_v = warp == kFetchVWarp;
        tree_fetch<T, QT, D, BS>(g, is_v, sh, q_tile, is_v ? v_tiles : k_tiles,
                                 raw_tiles + (is_v ? kRawStages * C::kRawBytes : 0), ok);
    } else if (warp == kMmaWarp) {
        // --- MMAs: the warp waits together, one lane issues ---------------------------------
        const uint32_t idesc_qk =
            umma_idesc(kBf16, false, kTreeRows, kTreeTile) | (p.negate ? kUmmaNegateA : 0);
        constexpr uint32_t kIdescPv =
            umma_idesc(std::is_same<PT, __nv_bfloat16>::value, true, kTreeRows, D);
        const auto wait_warp = [&](uint64_t &bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, wait(bar, parity));
            return ok;
        };
        int pending = -1; // tile whose P V is still to be issued
        bool pending_first = false, last = false;
        int segments_read = 0;
        uint32_t q_at = q_tile;
        const auto issue_pv = [&]() {
            const int st = pending % NS;
            if (!wait_warp(sh.p_full[pending & 1], (pending >> 1) & 1) ||
                !wait_warp(sh.v_full[st], (pending / NS) & 1))
                return;
            bool add = !pending_first;
            if (pending_first) {
                if (segments_read > 0 && !wait_warp(sh.o_free, (segments_read - 1) & 1))
                    return;
                ++segments_read;
                add = *(volatile int32_t *)&sh.keep_o == pending;
            }
            tcgen05_fence_after();
            const uint64_t v = umma_desc(v_tiles + st * C::kTileBytes, 1024, C::kGroupBytes);
            const uint32_t a = tmem + C::kS0 + (pending & 1) * kTreeTile;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kTreeTile / 16; ++k)
                    tcgen05_mma_ts(tmem, a + k * 8, v + (k * 2 * C::kGroupBytes >> 4), kIdescPv,
                                   add || k > 0);
                tcgen05_commit(smem_addr(&sh.v_empty[st]));
                tcgen05_commit(smem_addr(&sh.o_full));
            }
            __syncwarp();
            pending = -1;
        };
        for (int it = 0, seg = -1, seg_end = 0; ok; ++it) {
            const bool first = it == seg_end;
            if (first) {
                if (last) {
                    if (pending >= 0)
                        issue_pv();
                    break;
                }
                ++seg;
                if (!wait_warp(sh.q_full[seg & 3], (seg >> 2) & 1))
                    break;
                const TreeSegment &d = sh.seg[seg & 3];
                seg_end = it + d.tile1 - d.tile0;
                last = d.last;
                q_at = q_tile + d.q_at;
            }
            const int st = it % NS;
            if (!wait_warp(sh.k_full[st], (it / NS) & 1))
                break;
            tcgen05_fence_after();
            const uint64_t q0 = umma_desc(q_at, 16, 1024);
            const uint64_t k0 = umma_desc(k_tiles + st * C::kTileBytes, 16, C::kGroupBytes);
            const uint32_t s_tile = tmem + C::kS0 + (it & 1) * kTreeTile;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tcgen05_mma_ss(s_tile, q0 + (((k / 4) * (kTreeRows * 128) + (k % 4) * 32) >> 4),
                                   k0 + (((k / 4) * 1024 + (k % 4) * 32) >> 4), idesc_qk, k > 0);
                tcgen05_commit(smem_addr(&sh.s_full[it & 1]));
                tcgen05_commit(smem_addr(&sh.k_empty[st]));
                if (it + 1 == seg_end)
                    tcgen05_commit(smem_addr(&sh.q_empty[seg & 1]));
            }
            __syncwarp();
            if (pending >= 0)
                issue_pv();
            pending = it;
            pending_first = first;
        }
        if (!ok) { // MMAs in flight read shared memory and write tensor memory
            if (elect_one())
                tcgen05_commit(smem_addr(&sh.drain));
            __syncwarp();
            mbar_wait_bounded(smem_addr(&sh.drain), 0, kWaitLimitNs);
        }
    } else if (warp < kSoftmaxWarps) {
        // --- softmax, one thread per row ----------------------------------------------------
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const uint32_t o_column = tmem + lanes;
        const float c = p.qk_scale_log2;
        // Every lane or none: what follows a wait is done by whole warps.
        const auto wait_warp = [&](uint64_t &bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, wait(bar, parity));
            return ok;
        };
        uint32_t syncs = 0; // of the softmax warps among themselves, bounded like all others
        const auto sync_warps = [&]() {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&sh.warps));
            return wait_warp(sh.warps, syncs++ & 1);
        };
        if (tid == 0) {
            // The unit that this piece begins inside of, if it was cut here first.
            const TreePlan &plan = sh.plan;
            const int piece = blockIdx.x >> (plan.stride - 1);
            TreeMergeRecord rec = {0, 0, 0, 0, 0};
            if (plan.tile > 0 && plan.piece(piece - 1) <= plan.unit_begin + kTreeUnitCost) {
                const TreeSeq &q = plan.q;
                const int64_t unit_last = plan.unit_begin + kTreeUnitCost + q.tiles - 1;
                int e = piece, hi = plan.pieces - 1; // the piece with the unit's last tile
                while (e < hi) {
                    const int mid = (e + hi + 1) / 2;
                    if (plan.piece(mid) <= unit_last)
                        e = mid;
                    else
                        hi = mid - 1;
                }
                const int per_tile = kTreeRows / p.group, row_tiles = q.row_tiles >> (plan.stride - 1);
                const int rt = plan.unit % row_tiles * plan.stride + plan.lane;
                rec.parts = e - piece + 2;
                rec.stride = plan.stride;
                rec.rows = min(per_tile, q.nodes - rt * per_tile) * p.group;
                rec.first_row = q.first + rt * per_tile;
                rec.kv_head = plan.unit / row_tiles;
            }
            p.ws_records[blockIdx.x] = rec;
        }
        __syncwarp();
        const int node = tid / p.group; // of the tile
        int it = 0;
        TreeSegment d, d_next; // this segment, and the next once it is known
        TreeSeen ahead;        // mask words of the next masked tile
        bool live = false;
        const int32_t *words = nullptr;
        const auto masked = [&](const TreeSegment &of, int tile) {
            return (tile + 1) * kTreeTile > of.ctx;
        };
        const auto look_ahead = [&](int seg) { // at segment seg, and its first tile's mask
            if (!wait_warp(sh.d_full[seg & 3], (seg >> 2) & 1))
                return;
            d_next = sh.seg[seg & 3];
            live = tid < d_next.rows;
            words = p.mask + (size_t)(d_next.row0 + (live ? node : 0)) * p.mask_words;
            if (live && masked(d_next, d_next.tile0))
                ahead.load(words, p.mask_words, d_next.tile0 * kTreeTile, d_next.ctx);
        };
        look_ahead(0);
        for (int seg = 0; ok; ++seg) {
            d = d_next;
            const bool warp_live = warp * 32 < d.rows, now_live = live;
            float m = -INFINITY, l = 0.f;
            float R = kTreeLeastR; // fp8: a power of two, O is in units of
            bool saw = false, poison = false;
            for (int tile = d.tile0; tile < d.tile1 && ok; ++tile, ++it) {
                const uint32_t s_column = tmem + lanes + C::kS0 + (it & 1) * kTreeTile;
                const int t0 = tile * kTreeTile, st = it % NS;
                const bool special = masked(d, tile); // uniform over the CTA
                uint64_t seen = ~0ull;
                if (special)
                    seen = live ? ahead.bits(t0, d.ctx, d.n) : 0ull;
                if (!wait_warp(sh.s_full[it & 1], (it >> 1) & 1))
                    break;
                tcgen05_fence_after();
                uint64_t strange = 0;
                if (special || tile + 1 == d.tile1) {
                    // V has to be here for what follows, and the fetching
                    // warp's word on its block ids with it.
                    if (!wait_warp(sh.v_full[st], (it / NS) & 1))
                        break;
                    poison = *(volatile int32_t *)&sh.poison[seg & 3] != 0;
                }
                constexpr int kPieces = D / 16;
                const int vj = tid >> 1; // this thread's row of V, and its pieces
                const uint32_t v_tile = v_tiles + st * C::kTileBytes;
                if (special) {
                    // Two threads a row of V: those of nodes, and behind the last
                    // token, are looked through.
                    bool bad = false;
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const uint32_t at =
                            v_tile + tree_piece_at<D>(vj, (tid & 1) * kPieces + i);
                        if (t0 + vj >= d.ctx) {
                            uint4 x;
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                         : "r"(at)
                                         : "memory");
                            bad |= not_finite<PT>(x);
                        }
                    }
                    if (bad)
                        atomicOr(&sh.strange[it & 1][vj >> 5], 1u << (vj & 31));
                    if (!sync_warps())
                        break;
                    strange = (uint64_t)*(volatile uint32_t *)&sh.strange[it & 1][1] << 32 |
                              *(volatile uint32_t *)&sh.strange[it & 1][0];
                }
                constexpr int NC = kTreeTile;
                uint32_t x[NC];
                float alpha = 1.f, keep = 1.f; // what O, and l, are multiplied by
                bool rescale = false;
                if (C::kFp8 && (!wait_warp(sh.ks_full[it & 3], (it >> 2) & 1) ||
                                !wait_warp(sh.vs_full[it & 3], (it >> 2) & 1)))
                    break;
                // Two bodies, so that tiles that every row sees whole carry
                // none of the masking.
                const auto softmax = [&](auto is_masked) {
                    constexpr bool kMasked = decltype(is_masked)::value;
#pragma unroll
                    for (int k = 0; k < NC; k += 32)
                        tmem_ld_x32(s_column + k, x + k);
                    float factor = c, log2_R = 0.f;
                    if constexpr (C::kFp8) {
                        const float4 *ks = reinterpret_cast<const float4 *>(sh.ks[it & 3]);
#pragma unroll
                        for (int k = 0; k < NC / 4; ++k) {
                            const float4 f = ks[k];
                            const float2 y = mul_f32x2(make_float2(__uint_as_float(x[4 * k]),
                                                                   __uint_as_float(x[4 * k + 1])),
                                                       make_float2(f.x, f.y));
                            const float2 z =
                                mul_f32x2(make_float2(__uint_as_float(x[4 * k + 2]),
                                                      __uint_as_float(x[4 * k + 3])),
                                          make_float2(f.z, f.w));
                            x[4 * k] = __float_as_uint(y.x);
                            x[4 * k + 1] = __float_as_uint(y.y);
                            x[4 * k + 2] = __float_as_uint(z.x);
                            x[4 * k + 3] = __float_as_uint(z.y);
                        }
                        factor = 1.f;
                        // Weights are p * scale / R, R the power of two
                        // above the largest size of a V scale so far, at
                        // least kTreeLeastR: in f16's range. 1 / R goes into
                        // the exponent.
                        float top_v = sh.vmax[it & 3];
                        if (kMasked) {
                            top_v = 0.f;
#pragma unroll 2
                            for (int k = 0; k < NC; k += 4) {
                                const float4 v =
                                    *reinterpret_cast<const float4 *>(&sh.vs[it & 3][k]);
                                const uint32_t b = (uint32_t)(seen >> k);
                                top_v = max3(top_v, fabsf(b & 1 ? v.x : 0.f),
                                             fabsf(b & 2 ? v.y : 0.f));
                                top_v = max3(top_v, fabsf(b & 4 ? v.z : 0.f),
                                             fabsf(b & 8 ? v.w : 0.f));
                            }
                        }
                        if (top_v > R) {
                            const float up2 = __uint_as_float(
                                min((__float_as_uint(top_v) + 0x7fffffu) & 0x7f800000u,
                                    0x7e800000u));
                            alpha = R / up2;
                            rescale = tile > d.tile0;
                            R = up2;
                        }
                        log2_R = (float)((int)(__float_as_uint(R) >> 23) - 127);
                    }
                    if (kMasked) {
#pragma unroll
                        for (int k = 0; k < NC; ++k)
                            if (!((seen >> k) & 1))
                                x[k] = __float_as_uint(-INFINITY);
                    }
                    saw |= !kMasked || seen != 0;
                    float mx[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx[k] = __uint_as_float(x[k]);
#pragma unroll
                    for (int k = 4; k < NC - 4; k += 2)
                        mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], __uint_as_float(x[k]),
                                                __uint_as_float(x[k + 1]));
                    mx[0] = max3(mx[0], __uint_as_float(x[NC - 4]), __uint_as_float(x[NC - 3]));
                    mx[1] = max3(mx[1], __uint_as_float(x[NC - 2]), __uint_as_float(x[NC - 1]));
                    mx[0] = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
                    const float top = !kMasked || seen != 0 ? mx[0] * factor : -INFINITY;
                    if (top > m + kTreeSlack || (m == -INFINITY && top > m)) {
                        keep = m == -INFINITY ? 0.f : ex2(m - top);
                        alpha *= keep;
                        rescale = tile > d.tile0;
                        m = top;
                    }
                    const float off = kTreeBias - (m == -INFINITY ? 0.f : m) - log2_R;
                    const float2 c2 = make_float2(factor, factor), off2 = make_float2(off, off);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int k = 0; k < NC / 2; ++k) {
                        float2 w = fma_f32x2(make_float2(__uint_as_float(x[2 * k]),
                                                         __uint_as_float(x[2 * k + 1])),
                                             c2, off2);
                        w.x = ex2(w.x);
                        w.y = ex2(w.y);
                        sum[k & 1] = add_f32x2(sum[k & 1], w);
                        if constexpr (C::kFp8) {
                            const float4 v4 =
                                reinterpret_cast<const float4 *>(sh.vs[it & 3])[k >> 1];
                            w = mul_f32x2(w, k & 1 ? make_float2(v4.z, v4.w)
                                                   : make_float2(v4.x, v4.y));
                        }
                        x[k] = pack2<PT>(w.x, w.y); // in place: pair k is done with x[2k..]
                    }
                    sum[0] = add_f32x2(sum[0], sum[1]);
                    const float more = sum[0].x + sum[0].y;
                    l = fmaf(l, keep, C::kFp8 ? more * R : more);
                };
                if (warp_live) {
                    if (special)
                        softmax(std::true_type{});
                    else
                        softmax(std::false_type{});
                }
                // O is complete up to the tile before.
                if (tile > d.tile0) {
                    if (!wait_warp(sh.o_full, (it - 1) & 1))
                        break;
                    tcgen05_fence_after();
                }
                if (warp_live) {
                    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld_x32(o_column + c0, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                            tmem_st_x32(o_column + c0, o);
                        }
                    }
                    tmem_st_x32(s_column, x);
                    tmem_wait_st();
                }
                if (strange) {
                    if (tile == d.tile0) {
                        uint32_t o[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = 0;
                        for (int c0 = 0; c0 < D; c0 += 32)
                            tmem_st_x32(o_column + c0, o);
                        tmem_wait_st();
                        if (tid == 0)
                            *(volatile int32_t *)&sh.keep_o = it;
                    }
                    if (warp_live) {
                        const int nodes = d.n - t0; // rows behind are just emptied
                        rescue_rows<PT, D>(nodes < 64 ? strange & ((1ull << nodes) - 1) : strange,
                                           seen, v_tile, s_column, o_column);
                    }
                    if (!sync_warps())
                        break;
                    if ((strange >> vj) & 1)
                        for (int i = 0; i < kPieces; ++i)
                            asm volatile(
                                "st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                    v_tile + tree_piece_at<D>(vj, (tid & 1) * kPieces + i)),
                                "r"(0)
                                : "memory");
                    if (tid < 2)
                        *(volatile uint32_t *)&sh.strange[it & 1][tid] = 0;
                    fence_proxy_async_smem();
                    if (!sync_warps())
                        break;
                }
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&sh.p_full[it & 1]));
                if (tile + 1 < d.tile1 && live && masked(d, tile + 1))
                    ahead.load(words, p.mask_words, t0 + kTreeTile, d.ctx);
            }
            // Before this segment's rows are written, for the latency.
            if (ok && !d.last)
                look_ahead(seg + 1);
            if (!ok || !wait_warp(sh.o_full, (it - 1) & 1))
                break;
            tcgen05_fence_after();
            if (warp_live) {
                // A row that saw nothing is zero; one that saw only scores of
                // minus infinity is NaN, as 0/0 is.
                const bool none = l == 0.f && !saw;
                if (d.slot < 0) {
                    const float inv = none ? 0.f : C::kFp8 ? R / l : 1.f / l;
                    const size_t at =
                        ((size_t)(d.row0 + node) * p.num_heads + d.kv_head * p.group +
                         (tid - node * p.group)) * D;
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld_x32(o_column + c0, o);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = __float_as_uint(poison ? NAN
                                                   : none ? 0.f
                                                          : __uint_as_float(o[k]) * inv);
                        if (now_live)
                            store_row32(p.out, p.out_dtype, at + c0, o);
                        __syncwarp();
                    }
                } else {
                    const size_t slot = (size_t)blockIdx.x * 2 + d.slot;
                    float4 *acc = p.ws_acc + slot * (D / 4) * kTreeRows + tid;
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld_x32(o_column + c0, o);
                        if (now_live) {
                            if constexpr (C::kFp8) {
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    o[k] = __float_as_uint(__uint_as_float(o[k]) * R);
                            }
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                __stcg(acc + (size_t)(c0 / 4 + k) * kTreeRows,
                                       make_float4(__uint_as_float(o[4 * k]),
                                                   __uint_as_float(o[4 * k + 1]),
                                                   __uint_as_float(o[4 * k + 2]),
                                                   __uint_as_float(o[4 * k + 3])));
                        }
                        __syncwarp();
                    }
                    if (now_live) // l = -0: the row saw only scores of minus infinity
                        __stcg(p.ws_ml + slot * kTreeRows + tid,
                               make_float2(m, poison ? NAN : l == 0.f && saw ? -0.f : l));
                }
            }
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&sh.o_free));
            if (d.last)
                break;
        }
    }
    if (!ok)
        report(p.dev_err, PA_DEVERR_TIMEOUT);
    tcgen05_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tcgen05_fence_after();
        tmem_dealloc(tmem, C::kColumns);
    }
}

// Joins the parts of the unit that is cut before CTA blockIdx.x + 1, if there
// is one and no earlier cut in it: O = sum_p 2^(m_p - M) acc_p / sum_p
// 2^(m_p - M) l_p. A thread has one row and kMergeCols columns of four; a unit
// in more than kMergeFew parts and of up to 32 (64) rows has four (two)
// threads a row, each with every fourth (second) part, whose sums meet in
// shared memory. Bound by the latency of its loads, a chunk of parts at a
// time, and by the number of CTAs that the launch brings: one 2000-token
// sequence of 8 K/V heads (up to 33 parts a unit) takes 13.0 us in all, 16.7
// with one thread a row and two columns each; blocks of 512 threads, which
// find no room beside the CTAs of the kernel before, 15.0.
constexpr int kMergeCols = 4, kMergeFew = 4;

struct TreeMergeSum {
    float m, l;
    float4 o[kMergeCols];
    bool saw;

    __device__ __forceinline__ void rescale(float to)
    {
        const float use = to == -INFINITY ? 0.f : to, keep = ex2(m - use);
        m = to;
        l *= keep;
#pragma unroll
        for (int k = 0; k < kMergeCols; ++k)
            o[k] = make_float4(o[k].x * keep, o[k].y * keep, o[k].z * keep, o[k].w * keep);
    }
};

template <int D>
__global__ void __launch_bounds__(kTreeRows) tree_merge_kernel(
    const __grid_constant__ TreeDecodeParams p)
{
    __shared__ TreeMergeSum other[96];
    pdl_launch_dependents();
    pdl_wait_prior_grid();
    const int b = blockIdx.x + 1;
    const TreeMergeRecord rec = p.ws_records[b];
    if (rec.parts == 0)
        return;
    // Threads of a group.
    const int span = rec.parts <= kMergeFew || rec.rows > 64 ? 128 : rec.rows > 32 ? 64 : 32;
    const int row = threadIdx.x % span, grp = threadIdx.x / span, groups = kTreeRows / span;
    const auto slot = [&](int i) {
        return i == 0 ? (size_t)(b - rec.stride) * 2 + 1 : (size_t)(b + (i - 1) * rec.stride) * 2;
    };
    constexpr int kChunk = 4; // parts whose loads are in flight together
    const int c0 = blockIdx.y * kMergeCols;
    TreeMergeSum sum;
    sum.m = -INFINITY;
    sum.l = 0.f;
    sum.saw = false;
#pragma unroll
    for (int k = 0; k < kMergeCols; ++k)
        sum.o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = grp; row < rec.rows && i0 < rec.parts; i0 += kChunk * groups) {
        float2 ml[kChunk];
        float4 a[kChunk][kMergeCols];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            ml[i] = make_float2(-INFINITY, 0.f);
            if (i0 + i * groups < rec.parts) {
                const size_t at = slot(i0 + i * groups);
                ml[i] = __ldcg(p.ws_ml + at * kTreeRows + row);
#pragma unroll
                for (int k = 0; k < kMergeCols; ++k)
                    a[i][k] = __ldcg(p.ws_acc + (at * (D / 4) + c0 + k) * kTreeRows + row);
            }
        }
        float top = sum.m;
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            top = fmaxf(top, ml[i].x);
        sum.rescale(top);
        const float use = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            if (i0 + i * groups >= rec.parts)
                break;
            const float w = ex2(ml[i].x - use);
            sum.saw |= ml[i].y != 0.f || signbit(ml[i].y);
            sum.l = fmaf(ml[i].y, w, sum.l);
#pragma unroll
            for (int k = 0; k < kMergeCols; ++k) {
                sum.o[k].x = fmaf(a[i][k].x, w, sum.o[k].x);
                sum.o[k].y = fmaf(a[i][k].y, w, sum.o[k].y);
                sum.o[k].z = fmaf(a[i][k].z, w, sum.o[k].z);
                sum.o[k].w = fmaf(a[i][k].w, w, sum.o[k].w);
            }
        }
    }
    if (groups > 1) {
        if (grp > 0)
            other[(int)threadIdx.x - span] = sum;
        __syncthreads();
        if (grp > 0)
            return;
        for (int g = 1; g < groups; ++g) {
            TreeMergeSum x = other[(g - 1) * span + row];
            const float top = fmaxf(sum.m, x.m);
            sum.rescale(top);
            x.rescale(top);
            sum.l += x.l;
            sum.saw |= x.saw;
#pragma unroll
            for (int k = 0; k < kMergeCols; ++k) {
                sum.o[k].x += x.o[k].x;
                sum.o[k].y += x.o[k].y;
                sum.o[k].z += x.o[k].z;
                sum.o[k].w += x.o[k].w;
            }
        }
    }
    if (row >= rec.rows)
        return;
    const bool none = sum.l == 0.f && !sum.saw;
    const float inv = none ? 0.f : 1.f / sum.l;
    const int node = row / p.group;
    const size_t at = ((size_t)(rec.first_row + node) * p.num_heads + rec.kv_head * p.group +
                       (row - node * p.group)) * D + c0 * 4;
#pragma unroll
    for (int k = 0; k < kMergeCols; ++k)
        store_row4(p.out, p.out_dtype, at + 4 * k,
                   make_float4(none ? 0.f : sum.o[k].x * inv, none ? 0.f : sum.o[k].y * inv,
                               none ? 0.f : sum.o[k].z * inv, none ? 0.f : sum.o[k].w * inv));
}

} // namespace pagedkv
