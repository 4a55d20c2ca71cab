"""Drafted trees over the paged cache on the GPU: masks, attention, acceptance
and compaction against plain 64-bit and integer forms, and a whole step."""
import numpy as np
import pytest
import torch

from tests.tree_cases import (TYPES, TreeBatch, accept_path, ancestors, fp8_bytes, pack_bits,
                              random_parents)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    import paged_kv_cache_417_b200
    return paged_kv_cache_417_b200


# --- attention -----------------------------------------------------------------------------------

EDGE_CTX = [0, 1, 7, 8, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 128, 129, 250]
EDGE_TREES = [1, 2, 5, 8, 0, 3, 13, 16, 17, 31, 32, 33, 4, 1, 6, 7, 20]


@pytest.mark.parametrize("cache,io", [("f16", "f16"), ("bf16", "bf16"), ("fp8", "f16"),
                                      ("fp8", "bf16")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [8, 16, 32])
def test_tree_decode_edge_lengths(pk, cache, io, dim, block):
    b = TreeBatch(1, EDGE_CTX, EDGE_TREES, kv_heads=2, group=4, dim=dim, block=block,
                  cache=cache, io=io, pad=3)
    b.check(b.decode(pk))


@pytest.mark.parametrize("kv_heads,group", [(1, 1), (3, 1), (1, 2), (2, 3), (5, 7), (1, 8), (2, 16),
                                            (1, 33), (1, 71), (1, 128)])
@pytest.mark.parametrize("cache", ["f16", "fp8"])
def test_tree_decode_head_layouts(pk, kv_heads, group, cache):
    b = TreeBatch(2, [40, 0, 77, 5], [6, 9, 1, 19], kv_heads=kv_heads, group=group, dim=64,
                  cache=cache)
    b.check(b.decode(pk))


@pytest.mark.parametrize("cache,io,dim", [("f16", "f16", 128), ("bf16", "bf16", 64),
                                          ("fp8", "bf16", 128)])
def test_tree_decode_any_mask(pk, cache, io, dim):
    """Any bits: rows that see nothing of the tree, bits past its end, and
    with no context rows that see nothing at all (zero rows)."""
    b = TreeBatch(3, [0, 0, 3, 50, 64, 130], [33, 7, 64, 40, 65, 9], dim=dim, cache=cache, io=io,
                  masks="any", words=4)
    b.check(b.decode(pk))
    b = TreeBatch(4, [0, 70], [12, 12], dim=dim, cache=cache, io=io, masks="none")
    out = b.decode(pk)
    b.check(out)
    assert not out[:12].any()


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cache", ["f16", "bf16"])
def test_tree_decode_output_types(pk, out_dtype, cache):
    b = TreeBatch(5, [19, 200], [8, 21], cache=cache, dim=128)
    b.check(b.decode(pk, out_dtype))


@pytest.mark.parametrize("trees,group", [([64, 1, 130], 4), ([300], 2), ([1024, 5], 1)])
def test_tree_decode_large_trees(pk, trees, group):
    b = TreeBatch(6, [90, 17, 3][:len(trees)], trees, kv_heads=1, group=group, dim=64)
    b.check(b.decode(pk))


@pytest.mark.parametrize("cache,io,dim,block", [("f16", "f16", 128, 16), ("bf16", "bf16", 128, 8),
                                                ("fp8", "f16", 64, 32), ("fp8", "bf16", 128, 16)])
def test_tree_decode_long_contexts(pk, cache, io, dim, block):
    """One sequence shared by many CTAs, beside short ones."""
    b = TreeBatch(7, [20011, 3, 700], [11, 4, 0], kv_heads=2, group=4, dim=dim, cache=cache,
                  io=io, block=block)
    b.check(b.decode(pk))


@pytest.mark.parametrize("kv_heads,group,n", [(8, 4, 40), (4, 1, 150), (1, 4, 700)])
def test_tree_decode_many_sequences(pk, kv_heads, group, n):
    rng = np.random.default_rng(n)
    b = TreeBatch(8, rng.integers(0, 150, n).tolist(), rng.integers(0, 9, n).tolist(),
                  kv_heads=kv_heads, group=group, dim=64)
    b.check(b.decode(pk))


@pytest.mark.parametrize("gain", [0.0, 8.0, 60.0])
@pytest.mark.parametrize("cache", ["f16", "bf16"])
def test_tree_decode_spread_of_scores(pk, gain, cache):
    """Equal scores, and maxima that move by hundreds from token to token."""
    b = TreeBatch(9, [500, 90], [9, 30], cache=cache, dim=128, q_gain=gain)
    b.check(b.decode(pk))


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_tree_decode_scales(pk, scale):
    b = TreeBatch(10, [150, 3], [9, 12], dim=64)
    b.check(b.decode(pk, scale=scale), scale=scale)


def test_tree_decode_rising_and_falling_scores(pk):
    """Keys that grow along the context (every tile has a new maximum), and
    that shrink."""
    for ends in ((0.0, 3.0), (3.0, 0.0)):
        b = TreeBatch(11, [600], [8], kv_heads=1, group=4, dim=64)
        ramp = torch.linspace(*ends, 608)
        for j in range(608):
            blk, off = int(b.table[0, j // 16]), j % 16
            b.pools[0][blk, :, off] = b.pools[0][blk, :, off] * ramp[j]
            b.pools[0][blk, :, off, 0] = ramp[j] * 10
        b.query[..., 0] = 6.0
        b.check(b.decode(pk))


def test_tree_decode_masked_nan_and_infinity(pk):
    """NaN and infinities in K and V rows of nodes: rows that do not attend to
    them are untouched, rows that do follow the arithmetic."""
    for cache, dim in (("f16", 64), ("bf16", 128), ("fp8", 128)):
        b = TreeBatch(12, [70, 0, 125], [40, 9, 20], dim=dim, cache=cache)
        def row(s, i, which):
            j = b.ctx[s] + i
            return int(b.table[s, j // 16]), j % 16, which
        def put(s, i, which, value):
            blk, off, w = row(s, i, which)
            if cache != "fp8":
                b.pools[w][blk, :, off, 3] = value
                b.pools[w][blk, :, off, dim - 1] = value
            else:  # the row's scale
                n = 16 * dim
                sc = b.pools[w][blk, :, n:].contiguous().view(torch.float32)
                sc[:, off] = value
                b.pools[w][blk, :, n:] = sc.view(torch.uint8)
        put(0, 5, 1, float("nan"))
        put(0, 30, 1, float("inf"))
        put(0, 7, 0, float("nan"))
        put(1, 4, 1, float("-inf"))
        put(2, 19, 1, float("nan"))
        put(2, 18, 0, float("nan"))
        b.check(b.decode(pk))


def test_tree_decode_nan_in_context_reaches_its_sequence_only(pk):
    b = TreeBatch(13, [70, 90], [5, 6], dim=64)
    b.pools[1][int(b.table[0, 1]), 0, 3, 7] = float("nan")
    b.check(b.decode(pk))


def test_tree_decode_leading_and_trailing_rows(pk):
    b = TreeBatch(14, [33, 5], [6, 3], lead=4, pad=9)
    b.check(b.decode(pk))


def test_tree_decode_without_trees(pk):
    b = TreeBatch(15, [40, 9], [0, 0], pad=3)
    b.check(b.decode(pk))


def test_tree_decode_repeats_bit_for_bit(pk):
    b = TreeBatch(16, [3000, 20, 900], [16, 5, 30], kv_heads=4, dim=128)
    first = b.decode(pk)
    for _ in range(3):
        assert torch.equal(b.decode(pk).nan_to_num(), first.nan_to_num())


def test_tree_decode_workspace_need_not_be_clean(pk):
    b = TreeBatch(17, [5000, 20], [16, 5], kv_heads=2, dim=64)
    q, k, *_ = b.cuda(pk)
    ws = pk.alloc_tree_workspace(k)
    ws.fill_(255)
    b.check(b.decode(pk, workspace=ws))


def test_tree_decode_bad_block_context_and_tree(pk):
    """Device-side refusals: error bits, NaN rows of that sequence, the
    others exact."""
    b = TreeBatch(18, [40, 60, 80], [5, 6, 7])
    want = b.expected()
    for bad in (-1, b.num_blocks, 2 ** 31 - 1):
        keep = int(b.table[1, 2])
        b.table[1, 2] = bad
        want[0][5:11] = float("nan")
        b.check(b.decode(pk, want_err=pk.PA_DEVERR_BLOCK_ID), expected=want)
        b.table[1, 2] = keep
    want = b.expected()
    want[0][5:11] = float("nan")
    for bad in (-1, -2 ** 31, 16 * b.table.shape[1] - 5, 2 ** 31 - 1):
        ctx, b.ctx = b.ctx, [40, bad, 80]
        b.check(b.decode(pk, want_err=pk.PA_DEVERR_CONTEXT_LEN), expected=want)
        b.ctx = ctx
    # Offsets: the second tree's end before its start; a tree past the rows.
    out = b.expected()[0]
    start = b.start.clone()
    for bad, lost in (([0, 5, 3, 18], [1]), ([-3, 5, 11, 18], [0]), ([0, 5, 11, 19], [2]),
                      ([0, 5, 11, 2 ** 31 - 1], [2])):
        b.start = torch.tensor(bad, dtype=torch.int32)
        q, k, v, table, ctx, st, mask = b.cuda(pk)
        got = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pk.tree_decode(got, q, k, v, table, ctx, st, mask, b.scale, dev_err=err)
        assert int(err.item()) == pk.PA_DEVERR_TREE
        for s, (a, e) in enumerate(((0, 5), (5, 11), (11, 18))):
            if s in lost:
                continue
            if bad == [0, 5, 3, 18]:
                if s == 2:
                    continue
                e = 3  # the third tree's rows begin inside the first one's
            assert (got[a:e].double().cpu() - out[a:e]).abs().max() < 4e-3
    b.start = start
    # A tree of more nodes than the mask has bits for.
    b = TreeBatch(19, [10, 20], [40, 5], words=1)
    got = b.decode(pk, want_err=pk.PA_DEVERR_TREE)
    assert torch.isnan(got[:40]).all() and torch.isfinite(got[40:]).all()


def test_tree_decode_graph_replays_with_other_lengths(pk):
    """One captured call; lengths, trees and tables change between replays."""
    batches = [TreeBatch(20 + i, ctx, tr, kv_heads=2, group=4, dim=64, words=2, spare_blocks=sp)
               for i, (ctx, tr, sp) in enumerate([([400, 3], [10, 30], 0), ([0, 90], [38, 2], 0),
                                                  ([900, 1], [1, 39], 0)])]
    nb = max(b.num_blocks for b in batches)
    width = max(b.table.shape[1] for b in batches)
    rows = 40
    q = torch.zeros(rows, 8, 64, dtype=torch.float16, device="cuda")
    k = torch.zeros(nb, 2, 16, 64, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
    start = torch.zeros(3, dtype=torch.int32, device="cuda")
    mask = torch.zeros(rows, 2, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    ws = pk.alloc_tree_workspace(k)
    call = lambda: pk.tree_decode(out, q, k, v, table, ctx, start, mask, 0.125, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for b in batches + batches[:1]:
        bq, bk, bv, bt, bc, bs, bm = b.cuda(pk)
        q[:b.rows], k[:b.num_blocks], v[:b.num_blocks] = bq, bk, bv
        table[:, :bt.shape[1]] = bt
        ctx.copy_(bc)
        start.copy_(bs)
        mask[:b.rows] = bm
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        b.check(out[:b.rows])


def test_tree_decode_on_two_streams(pk):
    """Two streams at once, a workspace each."""
    a = TreeBatch(24, [3000, 50], [16, 9], kv_heads=2, dim=128)
    b = TreeBatch(25, [10, 2000], [30, 12], kv_heads=2, dim=128)
    sides = []
    for x in (a, b):
        q, k, v, table, ctx, start, mask = x.cuda(pk)
        sides.append((torch.cuda.Stream(), torch.full_like(q, float("nan")), q, k, v, table, ctx,
                      start, mask, pk.alloc_tree_workspace(k)))
    torch.cuda.synchronize()
    for _ in range(5):
        for st, out, *rest, ws in sides:
            with torch.cuda.stream(st):
                pk.tree_decode(out, *rest, a.scale, workspace=ws)
    torch.cuda.synchronize()
    a.check(sides[0][1])
    b.check(sides[1][1])


@pytest.mark.parametrize("cache", ["f16", "fp8"])
def test_tree_decode_blocks_past_32_bit_offsets(pk, cache):
    """A pool of more than 2^32 bytes (2^31 elements), its last blocks in use."""
    b = TreeBatch(26, [100, 30], [7, 9], kv_heads=8, group=2, dim=128, cache=cache)
    per_block = b.pools[0][0].numel() * b.pools[0].element_size()
    total = (5 << 30) // per_block
    shift = total - b.num_blocks
    pools = []
    for x in b.pools:
        big = torch.empty(total, *x.shape[1:], dtype=x.dtype, device="cuda")
        big[shift:] = x.cuda()
        pools.append(big)
    q, _, _, table, ctx, start, mask = b.cuda(pk)
    table = torch.where(table >= 0, table + shift, table)
    if cache == "fp8":
        pools = [pk.Fp8Cache(x, b.block, b.dim, b.io) for x in pools]
    out = torch.full_like(q, float("nan"))
    pk.tree_decode(out, q, *pools, table, ctx, start, mask, b.scale)
    torch.cuda.synchronize()
    b.check(out)


def test_tree_decode_of_one_node_is_decode(pk):
    """A tree of one node is what pa_decode computes over one more token."""
    b = TreeBatch(27, [77, 3, 640], [1, 1, 1], kv_heads=2, group=4, dim=128)
    q, k, v, table, ctx, start, mask = b.cuda(pk)
    out, ref = torch.empty_like(q), torch.empty(q.shape, dtype=torch.float32, device="cuda")
    pk.tree_decode(out, q, k, v, table, ctx, start, mask, b.scale)
    pk.decode(ref, q, k, v, table, ctx + 1, 641, b.scale)
    assert (out.float() - ref).abs().max() < 4e-3


# --- masks ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("sizes,words,shape", [
    ([1], 1, "bushy"), ([8], 1, "chain"), ([32, 1, 0, 31], 1, "bushy"), ([33, 64], 2, "chain"),
    ([5, 100, 256], 8, "bushy"), ([256, 255], 8, "chain"), ([1024, 1000], 32, "chain"),
    ([1024, 3], 32, "bushy"), ([7, 600], 32, "star"), ([4] * 500, 1, "bushy")])
def test_tree_mask(pk, sizes, words, shape):
    rng = np.random.default_rng(len(sizes) + words)
    lead, pad = 2, 3
    start = torch.tensor([lead] + sizes).cumsum(0).to(torch.int32)
    rows = int(start[-1]) + pad
    parents = torch.full((rows,), 77, dtype=torch.int32)
    want = np.full((rows, words), -9, dtype=np.int32)
    depth = np.full(rows, -9, dtype=np.int32)
    for s, n in enumerate(sizes):
        a = int(start[s])
        p = random_parents(rng, n, shape)
        parents[a:a + n] = torch.tensor(p, dtype=torch.int32)
        anc = ancestors(p)
        want[a:a + n] = pack_bits(anc, words)
        depth[a:a + n] = anc.sum(1) - 1
    mask = torch.full((rows, words), -9, dtype=torch.int32, device="cuda")
    dep = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.tree_mask(mask, dep, parents.cuda(), start.cuda(), dev_err=err)
    assert int(err.item()) == 0
    assert np.array_equal(mask.cpu().numpy(), want)
    assert np.array_equal(dep.cpu().numpy(), depth)
    mask.fill_(-9)
    pk.tree_mask(mask, None, parents.cuda(), start.cuda())
    assert np.array_equal(mask.cpu().numpy(), want)


def test_tree_mask_bad_parents_and_trees(pk):
    # Node 1 names a later node, node 3 itself, node 4 something below -1: roots. Several
    # roots are allowed.
    parents = torch.tensor([-1, 2, 0, 3, -2, -1, 2], dtype=torch.int32)
    clean = [-1, -1, 0, -1, -1, -1, 2]
    mask = torch.zeros(7, 1, dtype=torch.int32, device="cuda")
    depth = torch.zeros(7, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 7], dtype=torch.int32)
    pk.tree_mask(mask, depth, parents.cuda(), start.cuda(), dev_err=err)
    assert int(err.item()) == pk.PA_DEVERR_TREE
    assert np.array_equal(mask.cpu().numpy(), pack_bits(ancestors(clean), 1))
    err.zero_()
    pk.tree_mask(mask, depth, torch.tensor(clean, dtype=torch.int32).cuda(), start.cuda(),
                 dev_err=err)
    assert int(err.item()) == 0
    # Bad offsets and a tree of more nodes than bits: left as they were.
    for offsets in ([0, 8], [-1, 7], [5, 3], [0, 33]):
        rows = 40 if offsets[1] == 33 else 7
        par = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        m = torch.full((rows, 1), 5, dtype=torch.int32, device="cuda")
        err.zero_()
        pk.tree_mask(m, None, par, torch.tensor(offsets, dtype=torch.int32).cuda(), dev_err=err)
        assert int(err.item()) == pk.PA_DEVERR_TREE and (m == 5).all()


# --- acceptance ----------------------------------------------------------------------------------

@pytest.mark.parametrize("sizes,max_path,shape,agree", [
    ([1, 0, 8], 4, "bushy", 0.8), ([5, 1, 0, 31], 16, "bushy", 0.9), ([64] * 40, 9, "bushy", 0.95),
    ([300, 1024, 2], 1024, "chain", 0.998), ([1024], 1024, "chain", 2.0), ([30, 7], 1, "chain", 2.0),
    ([257, 90], 12, "star", 0.9), ([3] * 300, 3, "bushy", 0.6)])
def test_tree_accept(pk, sizes, max_path, shape, agree):
    rng = np.random.default_rng(sum(sizes))
    lead, pad = 1, 2
    start = torch.tensor([lead] + sizes).cumsum(0).to(torch.int32)
    rows = int(start[-1]) + pad
    parents = np.full(rows, 50, dtype=np.int32)
    draft = rng.integers(0, 6, rows) + (1 << 40)  # few tokens: siblings that are alike
    target = rng.integers(0, 6, rows) + (1 << 40)
    want, lens, after = [], [], []
    for s, n in enumerate(sizes):
        a = int(start[s])
        p = random_parents(rng, n, shape)
        parents[a:a + n] = p
        for c in rng.permutation(n):
            if p[c] >= 0 and rng.random() < agree:
                target[a + p[c]] = draft[a + c]
        path, nxt = accept_path(p, draft[a:a + n].tolist(), target[a:a + n].tolist(), max_path)
        want.append(path + [-1] * (max_path - len(path)))
        lens.append(len(path))
        after.append(nxt)
    S = len(sizes)
    acc = torch.full((S, max_path), -9, dtype=torch.int32, device="cuda")
    al = torch.full((S,), -9, dtype=torch.int32, device="cuda")
    nt = torch.full((S,), -9, dtype=torch.int64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.tree_accept(acc, al, nt, torch.from_numpy(parents).cuda(), start.cuda(),
                   torch.from_numpy(draft).cuda(), torch.from_numpy(target).cuda(), dev_err=err)
    assert int(err.item()) == 0
    assert al.tolist() == lens and nt.tolist() == after
    assert acc.tolist() == want


def test_tree_accept_bad_trees(pk):
    dev = "cuda"
    tok = torch.zeros(6, dtype=torch.int64, device=dev)
    acc = torch.zeros(1, 4, dtype=torch.int32, device=dev)
    al = torch.zeros(1, dtype=torch.int32, device=dev)
    nt = torch.zeros(1, dtype=torch.int64, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    par = torch.tensor([-1, 0, 5, 2, -7, 1], dtype=torch.int32, device=dev)
    pk.tree_accept(acc, al, nt, par, torch.tensor([0, 6], dtype=torch.int32, device=dev), tok, tok,
                   dev_err=err)
    # Nodes 2 and 4 have bad parents and are no one's children; 0 -> 1 -> 5.
    assert int(err.item()) == pk.PA_DEVERR_TREE and acc.tolist() == [[0, 1, 5, -1]]
    for offsets in ([0, 7], [3, 2], [-1, 4]):
        err.zero_()
        pk.tree_accept(acc, al, nt, par, torch.tensor(offsets, dtype=torch.int32, device=dev), tok,
                       tok, dev_err=err)
        assert int(err.item()) == pk.PA_DEVERR_TREE
        assert al.tolist() == [0] and nt.tolist() == [-1] and acc.tolist() == [[-1] * 4]


# --- compaction ----------------------------------------------------------------------------------

def _pools(cache, layers, blocks, heads, block, dim, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(2 * layers):
        if cache == "fp8":
            x = torch.randint(0, 256, (blocks, heads, block * dim + 4 * block), generator=g,
                              device="cuda", dtype=torch.uint8)
        else:
            x = torch.randint(-2 ** 15, 2 ** 15, (blocks, heads, block, dim), generator=g,
                              device="cuda", dtype=torch.int16).view(TYPES[cache])
        out.append(x)
    return out


def _moved(pools, cache, block, dim, table, ctx, paths):
    """The pools after the moves, row by row in ascending order, as bytes."""
    out = []
    for x in pools:
        y = x.cpu().clone()
        if cache == "fp8":
            n = block * dim
            codes = y[..., :n].reshape(*y.shape[:2], block, dim).clone()
            scale = y[..., n:].reshape(*y.shape[:2], block, 4).clone()
            parts = [codes, scale]
        else:
            parts = [y.view(torch.int16)]
        for s, path in enumerate(paths):
            for k, node in enumerate(path):
                a, b = ctx[s] + node, ctx[s] + k
                for part in parts:
                    part[table[s][b // block], :, b % block] = \
                        part[table[s][a // block], :, a % block].clone()
        out.append(torch.cat([codes.flatten(2), scale.flatten(2)], -1) if cache == "fp8"
                   else parts[0])
    return out


@pytest.mark.parametrize("cache", ["f16", "bf16", "fp8"])
@pytest.mark.parametrize("dim,block,heads,layers", [(64, 8, 3, 2), (128, 16, 8, 1), (64, 32, 1, 5),
                                                    (128, 8, 2, 40)])
def test_tree_compact(pk, cache, dim, block, heads, layers):
    rng = np.random.default_rng(dim + layers)
    ctx = [0, 1, block - 1, block, 3 * block + 5, 40, 9]
    sizes = [1, 9, 33, 64, 0, 50, 7]
    paths = []
    for n in sizes:
        k = int(rng.integers(1, min(n, 20) + 1)) if n else 0
        paths.append(sorted(rng.permutation(n)[:k].tolist()))
    paths[5] = list(range(12))  # in place already
    need = [-(-(c + n) // block) for c, n in zip(ctx, sizes)]
    ids = rng.permutation(sum(need) + 2).tolist()
    table = np.full((len(ctx), max(need)), -1, dtype=np.int32)
    for s, k in enumerate(need):
        table[s, :k], ids = ids[:k], ids[k:]
    pools = _pools(cache, layers, sum(need) + 2, heads, block, dim, 3)
    want = _moved(pools, cache, block, dim, table.tolist(), ctx, paths)
    width = 24
    acc = torch.tensor([p + [-1] * (width - len(p)) for p in paths], dtype=torch.int32).cuda()
    lens = torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
    wrap = (lambda x: pk.Fp8Cache(x, block, dim)) if cache == "fp8" else (lambda x: x)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.tree_compact([wrap(x) for x in pools[0::2]], [wrap(x) for x in pools[1::2]],
                    torch.from_numpy(table).cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
                    acc, lens, dev_err=err)
    assert int(err.item()) == 0
    for x, y in zip(pools, want):
        got = x.cpu() if cache == "fp8" else x.cpu().view(torch.int16)
        assert torch.equal(got, y)


def test_tree_compact_long_path(pk):
    """A chain of 1024 nodes with one dropped near the front: every row moves by one."""
    n, block = 1024, 16
    pools = _pools("f16", 1, 70, 2, block, 64, 5)
    table = np.arange(66, dtype=np.int32)[None, ::-1].copy()
    path = [i for i in range(n) if i != 1]
    want = _moved(pools, "f16", block, 64, table.tolist(), [5], [path])
    acc = torch.tensor([path + [-1]], dtype=torch.int32).cuda()
    pk.tree_compact([pools[0]], [pools[1]], torch.from_numpy(table).cuda(),
                    torch.tensor([5], dtype=torch.int32).cuda(), acc,
                    torch.tensor([n - 1], dtype=torch.int32).cuda())
    for x, y in zip(pools, want):
        assert torch.equal(x.cpu().view(torch.int16), y)


def test_tree_compact_refuses_on_the_device(pk):
    block = 16
    good = [0, 3, 4]
    cases = [([[0, 3, 2]], [3], [20], "TREE"), ([[0, 0, 2]], [3], [20], "TREE"),
             ([[-1, 1, 2]], [3], [20], "TREE"), ([good], [4], [20], "TREE"),
             ([good], [-1], [20], "TREE"), ([good], [3], [-1], "CONTEXT_LEN"),
             ([good], [3], [44], "CONTEXT_LEN"), ([[0, 3, 2 ** 31 - 1]], [3], [20], "CONTEXT_LEN"),
             ([good], [3], [2 ** 31 - 1], "CONTEXT_LEN")]
    for paths, lens, ctx, bit in cases:
        pools = _pools("f16", 2, 6, 2, block, 64, 6)
        before = [x.clone() for x in pools]
        table = torch.tensor([[2, 5, 1]], dtype=torch.int32).cuda()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pk.tree_compact(pools[0::2], pools[1::2], table, torch.tensor(ctx, dtype=torch.int32).cuda(),
                        torch.tensor(paths, dtype=torch.int32).cuda(),
                        torch.tensor(lens, dtype=torch.int32).cuda(), dev_err=err)
        assert int(err.item()) == getattr(pk, "PA_DEVERR_" + bit), (paths, lens, ctx)
        for x, y in zip(pools, before):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    # A bad block: that row stays, the other moves.
    pools = _pools("f16", 1, 6, 2, block, 64, 7)
    want = _moved(pools, "f16", block, 64, [[2, 5, 0]], [14], [[0, 1, 5]])
    table = torch.tensor([[2, 5, 99]], dtype=torch.int32).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.tree_compact([pools[0]], [pools[1]], table, torch.tensor([14], dtype=torch.int32).cuda(),
                    torch.tensor([[0, 1, 5, 20]], dtype=torch.int32).cuda(),
                    torch.tensor([4], dtype=torch.int32).cuda(), dev_err=err)
    assert int(err.item()) == pk.PA_DEVERR_BLOCK_ID
    for x, y in zip(pools, want):
        assert torch.equal(x.cpu().view(torch.int16), y)


# --- a whole step --------------------------------------------------------------------------------

@pytest.mark.parametrize("cache", ["f16", "fp8"])
def test_speculative_steps_keep_the_cache_of_plain_decoding(pk, cache):
    """Several steps of drafting, masking, writing, attending, accepting and
    compacting, the block manager reserving and truncating: after each the
    cached rows are those of the kept tokens in order, and a decode over them
    is what it is over a cache that held them from the start."""
    from paged_kv_cache_417_b200.block_manager import BlockManager

    rng = np.random.default_rng(11)
    layers, kvh, group, dim, block = 2, 2, 4, 64, 16
    H, vocab = kvh * group, 50
    bm = BlockManager(64, block, rng.permutation(64))
    io = torch.float16

    def empty():
        if cache == "fp8":
            x = pk.Fp8Cache.empty(64, kvh, block, dim, io)
            x.data.zero_()
            return x
        return torch.zeros(64, kvh, block, dim, dtype=io, device="cuda")

    keys, values = [empty() for _ in range(layers)], [empty() for _ in range(layers)]
    # A token's rows depend on the token, its position and the layer alone.
    def rows_of(tokens, positions, layer, which):
        out = []
        for t, p in zip(tokens, positions):
            g = torch.Generator().manual_seed(int(t) * 7919 + int(p) * 31 + layer * 2 + which)
            out.append(torch.randn(kvh, dim, generator=g))
        return torch.stack(out).to(io).cuda()

    def write(tokens, positions, slots):
        for l in range(layers):
            pk.write_kv(rows_of(tokens, positions, l, 0), rows_of(tokens, positions, l, 1),
                        torch.as_tensor(slots).cuda(), keys[l], values[l])

    text = {}
    for s, n in enumerate([5, 16, 31]):
        bm.add_sequence(s)
        step = bm.prepare_tree([s], [n], 8)
        text[s] = rng.integers(0, vocab, n).tolist()
        write(text[s], range(n), step["slot_mapping"])
    # A sibling shares the last block of sequence 2, which must survive the trees.
    bm.fork(2, 9)
    shared = bm.block_table(9)
    sibling = [x.data.clone() if cache == "fp8" else x.clone() for x in (keys[0], values[1])]
    last = {s: int(rng.integers(0, vocab)) for s in text}
    for round_ in range(4):
        seqs = [0, 1, 2]
        sizes = [int(rng.integers(1, 14)) for _ in seqs]
        step = bm.prepare_tree(seqs, sizes, 8)
        dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in step.items()}
        if len(step["copy_pairs"]):
            pk.copy_blocks(keys, values, dev["copy_pairs"])
        N = sum(sizes)
        parents = sum((random_parents(rng, n) for n in sizes), [])
        par = torch.tensor(parents, dtype=torch.int32).cuda()
        mask = torch.empty(N, 1, dtype=torch.int32, device="cuda")
        depth = torch.empty(N, dtype=torch.int32, device="cuda")
        pk.tree_mask(mask, depth, par, dev["tree_start"])
        draft = rng.integers(0, vocab, N)
        for s in seqs:
            draft[step["tree_start"][s]] = last[s]
        seq_of = np.repeat(seqs, sizes)
        pos = depth.cpu().numpy() + step["context_lens"][seq_of]
        write(draft, pos, step["slot_mapping"])
        query = torch.randn(N, H, dim, device="cuda", dtype=io)
        outs = []
        for l in range(layers):
            out = torch.empty_like(query)
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            pk.tree_decode(out, query, keys[l], values[l], dev["block_tables"],
                           dev["context_lens"], dev["tree_start"], mask, dim ** -0.5, dev_err=err)
            assert int(err.item()) == 0
            outs.append(out)
        target = rng.integers(0, vocab, N)
        for c in rng.permutation(N):
            s = seq_of[c]
            if parents[c] >= 0 and rng.random() < 0.8:
                target[step["tree_start"][s] + parents[c]] = draft[c]
        acc = torch.empty(3, 8, dtype=torch.int32, device="cuda")
        lens = torch.empty(3, dtype=torch.int32, device="cuda")
        nxt = torch.empty(3, dtype=torch.int64, device="cuda")
        pk.tree_accept(acc, lens, nxt, par, dev["tree_start"], torch.from_numpy(draft).cuda(),
                       torch.from_numpy(target).cuda())
        pk.tree_compact(keys, values, dev["block_tables"], dev["context_lens"], acc, lens)
        for s in seqs:
            path = acc[s, :int(lens[s])].tolist()
            a = step["tree_start"][s]
            text[s] += [int(draft[a + i]) for i in path]
            bm.truncate(s, len(text[s]))
            assert bm.num_tokens(s) == len(text[s])
            last[s] = int(nxt[s])
            # The attention of the path's last node, from a cache built afresh.
            n = len(text[s])
            fresh_k, fresh_v = empty(), empty()
            slots = torch.arange(n, device="cuda")
            for l in range(layers):
                pk.write_kv(rows_of(text[s], range(n), l, 0), rows_of(text[s], range(n), l, 1),
                            slots, fresh_k, fresh_v)
                bt = torch.arange(8, dtype=torch.int32, device="cuda")[None]
                ref = torch.empty(1, H, dim, device="cuda")
                got = torch.empty(1, H, dim, device="cuda")
                q = query[a + path[-1]][None].contiguous()
                ln = torch.tensor([n], dtype=torch.int32, device="cuda")
                pk.decode(ref, q, fresh_k, fresh_v, bt, ln, n, dim ** -0.5)
                mine = torch.full((1, 8), -1, dtype=torch.int32)
                tb = bm.block_table(s)
                mine[0, :len(tb)] = torch.tensor(tb, dtype=torch.int32)
                pk.decode(got, q, keys[l], values[l], mine.cuda(), ln, n, dim ** -0.5)
                assert torch.equal(got, ref)  # the same rows in the same order
                assert (outs[l][a + path[-1]].float() - ref[0]).abs().max() < 4e-3
    for x, y in zip((keys[0], values[1]), sibling):
        x = x.data if cache == "fp8" else x
        rows = x[shared[-1]] if cache == "fp8" else x[shared[-1]]
        assert torch.equal(rows.view(torch.uint8), y[shared[-1]].view(torch.uint8))


def test_whole_step_in_one_graph(pk):
    """Mask, write, attention, acceptance and compaction captured once and
    replayed on other inputs."""
    rng = np.random.default_rng(3)
    S, N, kvh, H, dim, block = 2, 20, 2, 8, 64, 16
    dev = "cuda"
    keys = [torch.randn(8, kvh, block, dim, device=dev, dtype=torch.float16) for _ in range(2)]
    values = [torch.randn(8, kvh, block, dim, device=dev, dtype=torch.float16) for _ in range(2)]
    table = torch.tensor([[0, 1, 2, 3], [4, 5, 6, 7]], dtype=torch.int32, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    st = dict(parents=torch.zeros(N, **i32), start=torch.zeros(S + 1, **i32),
              ctx=torch.zeros(S, **i32), slots=torch.full((N,), -1, dtype=torch.int64, device=dev),
              draft=torch.zeros(N, dtype=torch.int64, device=dev),
              target=torch.zeros(N, dtype=torch.int64, device=dev),
              q=torch.zeros(N, H, dim, dtype=torch.float16, device=dev),
              k=torch.zeros(N, kvh, dim, dtype=torch.float16, device=dev),
              v=torch.zeros(N, kvh, dim, dtype=torch.float16, device=dev))
    mask, depth = torch.zeros(N, 1, **i32), torch.zeros(N, **i32)
    out = torch.zeros(2, N, H, dim, dtype=torch.float16, device=dev)
    acc, lens = torch.zeros(S, 6, **i32), torch.zeros(S, **i32)
    nxt = torch.zeros(S, dtype=torch.int64, device=dev)
    ws = pk.alloc_tree_workspace(keys[0])

    def step():
        pk.tree_mask(mask, depth, st["parents"], st["start"])
        for l in range(2):
            pk.write_kv(st["k"], st["v"], st["slots"], keys[l], values[l])
            pk.tree_decode(out[l], st["q"], keys[l], values[l], table, st["ctx"], st["start"],
                           mask, 0.125, workspace=ws)
        pk.tree_accept(acc, lens, nxt, st["parents"], st["start"], st["draft"], st["target"])
        pk.tree_compact(keys, values, table, st["ctx"], acc, lens)

    def fill(seed, sizes, ctx):
        g = torch.Generator().manual_seed(seed)
        start = np.cumsum([0] + sizes)
        par = sum((random_parents(rng, n) for n in sizes), [])
        st["parents"][:len(par)] = torch.tensor(par, dtype=torch.int32).to(dev)
        st["start"].copy_(torch.tensor(start, dtype=torch.int32))
        st["ctx"].copy_(torch.tensor(ctx, dtype=torch.int32))
        slots = torch.full((N,), -1, dtype=torch.int64)
        for s, n in enumerate(sizes):
            for i in range(n):
                j = ctx[s] + i
                slots[start[s] + i] = int(table[s, j // block]) * block + j % block
        st["slots"].copy_(slots)
        st["draft"].copy_(torch.randint(0, 3, (N,), generator=g))
        st["target"].copy_(torch.randint(0, 3, (N,), generator=g))
        for n in "qkv":
            st[n].copy_(torch.randn(st[n].shape, generator=g))

    fill(1, [8, 12], [20, 3])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    base = [x.clone() for x in keys + values]
    for seed, sizes, ctx in ((2, [5, 15], [40, 9]), (3, [0, 1], [7, 50]), (4, [20, 0], [0, 11])):
        fill(seed, sizes, ctx)
        res = []
        for how in (step, graph.replay):
            for x, y in zip(keys + values, base):
                x.copy_(y)
            out.zero_()
            how()
            torch.cuda.synchronize()
            res.append([x.clone() for x in (out, acc, lens, nxt, *keys, *values)])
        for x, y in zip(*res):
            assert torch.equal(x, y)


@pytest.mark.parametrize("cache,trees,group,dim", [
    ("f16", [64, 50, 0, 33], 4, 64),     # two row tiles each (of 128 rows)
    ("bf16", [120, 64, 100], 4, 128),    # four, two and four
    ("fp8", [40, 64], 4, 128), ("f16", [64, 20], 4, 64), ("f16", [96, 64], 4, 64)])
def test_tree_decode_row_tiles_in_pairs(pk, cache, trees, group, dim):
    """Trees that all have an even number of row tiles, which two CTAs share,
    and some of an odd number among them, split over many CTAs and not."""
    for ctx in ([30, 400, 70, 1][:len(trees)], [9000, 3000, 5, 2500][:len(trees)]):
        b = TreeBatch(28, ctx, trees, kv_heads=2, group=group, dim=dim, cache=cache)
        b.check(b.decode(pk))


# --- the binding's refusals, and odd but allowed calls --------------------------------------------

def test_binding_refuses_wrong_tensors(pk):
    i32 = dict(dtype=torch.int32, device="cuda")
    b = TreeBatch(29, [20, 3], [4, 5])
    q, k, v, table, ctx, start, mask = b.cuda(pk)
    out, ws = torch.empty_like(q), pk.alloc_tree_workspace(k)
    good = dict(out=out, query=q, key_cache=k, value_cache=v, block_tables=table,
                context_lens=ctx, tree_start=start, mask=mask, scale=np.float32(0.125),
                workspace=ws)
    pk.tree_decode(**good)
    for bad in (dict(out=out[:-1]), dict(out=out.double()), dict(out=out.transpose(0, 1)),
                dict(query=q.bfloat16()), dict(query=q[..., :32]), dict(query=q.cpu()),
                dict(query=q[:, ::2]), dict(value_cache=v[:-1]), dict(value_cache=v.bfloat16()),
                dict(key_cache=k.transpose(1, 2)), dict(block_tables=table.long()),
                dict(block_tables=table[0]), dict(block_tables=table[:1]),
                dict(block_tables=table.t()), dict(context_lens=ctx[:1]),
                dict(context_lens=ctx.long()), dict(tree_start=start[:2]),
                dict(tree_start=start[:0]), dict(tree_start=start.cpu()), dict(mask=mask[1:]),
                dict(mask=mask[:, 0]), dict(workspace=ws[:-16].cpu()),
                dict(dev_err=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            pk.tree_decode(**{**good, **bad})
    for bad in (dict(workspace=ws[:-16]), dict(workspace=ws[1:]),
                dict(scale=float("nan"))):
        with pytest.raises(pk.PagedKVError):
            pk.tree_decode(**{**good, **bad})
    par = torch.tensor([-1, 0, 0, 1], **i32)
    st = torch.tensor([0, 4], **i32)
    m, d = torch.zeros(4, 1, **i32), torch.zeros(4, **i32)
    for args in ((m[:3], d, par, st), (m, d[:3], par, st), (m.long(), d, par, st),
                 (m, d, par.long(), st), (m, d, par[::2], st), (m.t(), d, par, st),
                 (m, d, par, st[:0]), (m, d, par[None], st), (m.cpu(), d, par, st)):
        with pytest.raises(ValueError):
            pk.tree_mask(*args)
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    acc, ln, nx = torch.zeros(1, 3, **i32), torch.zeros(1, **i32), tok[:1].clone()
    for args in ((acc[0], ln, nx, par, st, tok, tok), (acc, ln.long(), nx, par, st, tok, tok),
                 (acc, ln, nx.int(), par, st, tok, tok), (acc, ln, nx, par, st, tok[:3], tok),
                 (acc, ln, nx, par, st, tok, tok.int())):
        with pytest.raises(ValueError):
            pk.tree_accept(*args)
    for kw in (dict(key_caches=[k, k[:-1]], value_caches=[v, v]),
               dict(value_caches=[]), dict(key_caches=[k.float()]), dict(value_caches=[v.bfloat16()]),
               dict(key_caches=[k.cpu()]), dict(accepted=acc[0]), dict(context_lens=ctx)):
        call = dict(key_caches=[k], value_caches=[v], block_tables=table[:1], context_lens=ctx[:1],
                    accepted=acc, accepted_lens=ln)
        call.update(kw)
        with pytest.raises(ValueError):
            pk.tree_compact(**call)


def test_calls_with_nothing_to_do(pk):
    """No sequences; sequences with empty trees and no rows; no block columns."""
    i32 = dict(dtype=torch.int32, device="cuda")
    none = torch.zeros(0, **i32)
    tok = torch.zeros(0, dtype=torch.int64, device="cuda")
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16, device="cuda")
    q = torch.zeros(0, 8, 64, dtype=torch.float16, device="cuda")
    for S in (0, 3):
        start = torch.zeros(S + 1, **i32)
        ctx = torch.full((S,), 7, **i32)
        pk.tree_mask(torch.zeros(0, 1, **i32), none, none, start)
        acc, ln = torch.full((S, 4), 9, **i32), torch.full((S,), 9, **i32)
        nx = torch.full((S,), 9, dtype=torch.int64, device="cuda")
        pk.tree_accept(acc, ln, nx, none, start, tok, tok)
        assert (acc == -1).all() and (ln == 0).all() and (nx == -1).all()
        err = torch.zeros(1, **i32)
        pk.tree_decode(q.clone(), q, k, k, torch.zeros(S, 1, **i32), ctx, start,
                       torch.zeros(0, 1, **i32), 0.1, dev_err=err)
        pk.tree_compact([k], [k.clone()], torch.zeros(S, 1, **i32), ctx, acc, ln, dev_err=err)
        assert int(err.item()) == 0
    # A tree, but no column in the table: NaN rows, as for any that does not fit.
    out = torch.zeros(2, 8, 64, dtype=torch.float16, device="cuda")
    err = torch.zeros(1, **i32)
    pk.tree_decode(out, torch.zeros_like(out), k, k, torch.zeros(1, 0, **i32),
                   torch.zeros(1, **i32), torch.tensor([0, 2], **i32), torch.zeros(2, 1, **i32), 0.1,
                   dev_err=err)
    assert int(err.item()) == pk.PA_DEVERR_CONTEXT_LEN and torch.isnan(out).all()


@pytest.mark.parametrize("seed", range(24))
def test_tree_decode_drawn_cases(pk, seed):
    """Shapes, lengths, masks and types drawn over their ranges."""
    rng = np.random.default_rng(1000 + seed)
    cache = ["f16", "bf16", "fp8"][seed % 3]
    kv, group = [(1, 8), (2, 4), (8, 1), (5, 7), (1, 33), (3, 2), (2, 16), (1, 1)][seed % 8]
    S = int(rng.integers(1, 7))
    top = int(2 ** rng.uniform(0, 11.5))
    ctx = [int(x) for x in rng.integers(0, top + 1, S)]
    trees = [int(x) for x in rng.integers(0, int(2 ** rng.uniform(0, 7.5)) + 1, S)]
    trees[0] = max(trees[0], 1)
    b = TreeBatch(seed, ctx, trees, kv_heads=kv, group=group, dim=[64, 128][seed // 2 % 2],
                  block=[8, 16, 32][seed // 3 % 3], cache=cache,
                  io=["f16", "bf16"][seed // 6 % 2] if cache == "fp8" else None,
                  masks=["tree", "any"][seed // 4 % 2], shape=["bushy", "chain"][seed // 5 % 2],
                  pad=int(rng.integers(0, 4)), q_gain=float(2 ** rng.uniform(-2, 3)),
                  words=None if seed % 2 else max(1, -(-max(trees) // 32)) + 1)
    scale = b.scale * float(rng.choice([1.0, 1.0, -1.0]))
    b.check(b.decode(pk, scale=scale), scale=scale)


@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_tree_decode_fp8_scales_of_any_size(pk, io):
    """Row scales from 2^-30 to 2^12 side by side, and rows of zeros."""
    b = TreeBatch(30, [150, 3], [10, 7], kv_heads=2, group=4, dim=64, cache="fp8", io=io)
    n = 16 * 64
    rng = np.random.default_rng(5)
    for which, (lo, hi) in ((0, (-3, 3)), (1, (-30, 12))):
        sc = b.pools[which][..., n:].contiguous().view(torch.float32)
        sc *= torch.from_numpy(2.0 ** rng.integers(lo, hi, sc.shape)).float()
        sc[::3, :, ::5] *= 0
        b.pools[which][..., n:] = sc.view(torch.uint8)
    b.check(b.decode(pk, torch.float32))


@pytest.mark.parametrize("cache,io,dim", [("f16", "f16", 128), ("bf16", "bf16", 64),
                                          ("fp8", "f16", 64), ("fp8", "bf16", 128)])
def test_tree_decode_odd_rows_in_the_second_masked_tile_only(pk, cache, io, dim):
    """Trees that cross a 64-token boundary, at most 64 rows each (two of the four
    softmax warps idle): V is finite in their first masked tile, and holds NaN behind
    the last token and an infinity in a node of the second one. Every call of many
    gives the same bits."""
    n = 60
    b = TreeBatch(31, [50 + i % 14 + 64 * (i % 3) for i in range(n)], [16] * n, kv_heads=4,
                  group=4, dim=dim, cache=cache, io=io)
    for s in range(0, n, 4):
        j = (b.ctx[s] + 15) // 64 * 64  # the first node of the second tile
        assert b.ctx[s] < j < b.ctx[s] + 16
        blk, off = int(b.table[s, j // 16]), j % 16
        if cache == "fp8":
            sc = b.pools[1][blk, :, 16 * dim:].contiguous().view(torch.float32)
            sc[:, off] = float("inf")
            b.pools[1][blk, :, 16 * dim:] = sc.view(torch.uint8)
        else:
            b.pools[1][blk, :, off, 5] = float("inf")
    q, k, v, table, ctx, start, mask = b.cuda(pk)
    ws = pk.alloc_tree_workspace(k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.full_like(q, float("nan")) for _ in range(20)]
    for _ in range(20):
        for o in outs:
            pk.tree_decode(o, q, k, v, table, ctx, start, mask, b.scale, workspace=ws, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for o in outs[1:]:
            assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
    b.check(outs[0])


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("powers", ["tiny", "subnormal", "tiny_first", "huge", "huge_first", "any"])
def test_tree_decode_fp8_extreme_value_scales(pk, io, dim, powers):
    """V scales down to the smallest number and up to 2^94 or so: alone, in the first
    64-token tile (and every later one ordinary, or the other way round), and mixed."""
    ctx = [150, 3, 700]
    b = TreeBatch(32, ctx, [10, 7, 9], kv_heads=2, group=4, dim=dim, cache="fp8", io=io)
    n = 16 * dim
    rng = np.random.default_rng(6)
    sc = b.pools[1][..., n:].contiguous().view(torch.float32)  # about 2^-7 each
    first = torch.zeros(sc.shape[0], dtype=torch.bool)
    for s in range(3):
        first[b.table[s, :4].long().clamp(min=0)] = True
    first = first[:, None, None]
    if powers == "tiny":
        sc *= 2.0 ** -110
    elif powers == "subnormal":
        sc *= 2.0 ** -70
        sc *= 2.0 ** -67
    elif powers == "tiny_first":
        sc = torch.where(first, sc * 2.0 ** -118, sc)
    elif powers == "huge":
        sc *= 2.0 ** 101
    elif powers == "huge_first":
        sc = torch.where(first, sc * 2.0 ** 101, sc * 2.0 ** -50)
    else:
        sc *= torch.from_numpy(2.0 ** rng.integers(-119, 101, sc.shape)).float()
    b.pools[1][..., n:] = sc.view(torch.uint8)
    got = b.decode(pk, torch.float32).double().cpu()
    want, room = b.expected()
    assert torch.isfinite(want).all() and torch.isfinite(got).all()
    # Beside the bound of expected(): p times a scale over a power of two of at least
    # 2^-104, times 2^8, is rounded to fp16, off by 2^-25 below its normal range; codes
    # are at most 448 < 2^9. Rounding the output: half a step of fp32.
    tokens = 709
    lim = room + tokens * 2.0 ** (-25 - 8 - 104 + 9) + (want.abs() + room) * 2.0 ** -24 + 2.0 ** -150
    assert ((got - want).abs() <= lim).all(), float(((got - want).abs() / lim).max())


def test_tree_decode_workspace_keeps_nothing(pk):
    """Every (m, l) pair of the workspace is this call's: rows that were not filled, as
    after a wait that ran out, hold l = NaN, which makes what is merged from them NaN."""
    b = TreeBatch(33, [5000, 20], [16, 5], kv_heads=2, dim=64)
    q, k, *_ = b.cuda(pk)
    ws = pk.alloc_tree_workspace(k)
    old = 1.0
    ws.view(torch.float32).fill_(old)
    b.check(b.decode(pk, workspace=ws))
    ctas = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    pairs = ws[-ctas * 2 * 128 * 8:]  # the workspace's last part
    l = pairs.view(torch.float32).reshape(ctas, 2, 128, 2)[..., 1]
    assert not (l == old).any()
    assert torch.isnan(l).any() and torch.isfinite(l).any()
    # One bad block in one part of a sequence that many CTAs share: NaN rows.
    b.table[0, 100] = b.num_blocks
    got = b.decode(pk, workspace=ws, want_err=pk.PA_DEVERR_BLOCK_ID)
    assert torch.isnan(got[:16]).all() and torch.isfinite(got[16:]).all()


@pytest.mark.parametrize("cache,layers", [("f16", 3), ("fp8", 3), ("bf16", 256)])
def test_tree_compact_caches_that_layers_share(pk, cache, layers):
    """A cache listed for several layers, or as K and V of one, is moved once."""
    block, dim, heads = 16, 64, 2
    pools = _pools(cache, 2, 8, heads, block, dim, 8)
    table, ctx = [[2, 5, 1], [7, 0, 3]], [3, 14]
    paths = [[0, 2, 3, 4, 7, 20], [1, 2, 3, 4, 5, 6, 7, 8]]
    want = _moved(pools, cache, block, dim, table, ctx, paths)
    acc = torch.tensor([p + [-1] * (8 - len(p)) for p in paths], dtype=torch.int32).cuda()
    lens = torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
    wrap = (lambda x: pk.Fp8Cache(x, block, dim)) if cache == "fp8" else (lambda x: x)
    a, b, c, d = map(wrap, pools)
    keys, values = [a, b, a], [c, d, d]
    if layers > 3:
        keys, values = [a, b] * (layers // 2), [b, c] * (layers // 2 - 1) + [d, d]
    pk.tree_compact(keys, values, torch.tensor(table, dtype=torch.int32).cuda(),
                    torch.tensor(ctx, dtype=torch.int32).cuda(), acc, lens)
    for x, y in zip(pools, want):
        got = x.cpu() if cache == "fp8" else x.cpu().view(torch.int16)
        assert torch.equal(got, y)


@pytest.mark.parametrize("dim,sign", [(64, "all"), (128, "all"), (64, "some"), (128, "some")])
def test_tree_decode_fp8_negative_scales(pk, dim, sign):
    """A row's values are its codes times its scale, whatever the scale's sign."""
    b = TreeBatch(34, [150, 3, 70], [10, 7, 9], kv_heads=2, group=4, dim=dim, cache="fp8")
    n = 16 * dim
    rng = np.random.default_rng(7)
    for which in (0, 1):
        sc = b.pools[which][..., n:].contiguous().view(torch.float32)
        if sign == "all":
            sc *= -1
        else:
            # The negative ones are the larger in size.
            neg = torch.from_numpy(rng.random(sc.shape) < 0.3)
            sc = torch.where(neg, -sc * (16 if which else 1), sc / (16 if which else 1))
        b.pools[which][..., n:] = sc.view(torch.uint8)
    b.check(b.decode(pk, torch.float32))
