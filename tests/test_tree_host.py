"""Drafted trees without a GPU: refusals before any launch, the block
manager's share, and the plain forms the GPU tests compare with."""
import ctypes
import resource

import numpy as np
import pytest
import torch

from tests.tree_cases import TreeBatch, accept_path, ancestors, pack_bits


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_417_b200
    return paged_kv_cache_417_b200


FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: checks fail first
ODD = ctypes.c_void_p(0x1008)


def test_mask_and_accept_refusals(pk):
    L = pk._lib
    def mask(m=FAKE, par=FAKE, start=FAKE, S=1, N=4, words=1):
        return L.pa_tree_mask(m, None, par, start, S, N, words, None, None)
    assert mask(S=-1) == pk.PA_ERR_INVALID_ARG
    assert mask(N=-1) == pk.PA_ERR_INVALID_ARG
    assert mask(S=65536) == pk.PA_ERR_UNSUPPORTED
    assert mask(words=0) == pk.PA_ERR_INVALID_ARG
    assert mask(words=33) == pk.PA_ERR_INVALID_ARG
    for name in ("m", "par", "start"):
        assert mask(**{name: None}) == pk.PA_ERR_INVALID_ARG
    assert mask(m=None, par=None, start=None, S=0) == pk.PA_OK

    def accept(path=4, S=1, N=4, ptrs=(FAKE,) * 7):
        return L.pa_tree_accept(*ptrs, S, N, path, None, None)
    assert accept(path=0) == pk.PA_ERR_INVALID_ARG
    assert accept(path=1025) == pk.PA_ERR_INVALID_ARG
    assert accept(S=-1) == pk.PA_ERR_INVALID_ARG
    assert accept(N=-1) == pk.PA_ERR_INVALID_ARG
    for i in range(7):
        assert accept(ptrs=(FAKE,) * i + (None,) + (FAKE,) * (6 - i)) == pk.PA_ERR_INVALID_ARG
    assert accept(S=0, ptrs=(None,) * 7) == pk.PA_OK


def test_decode_refusals(pk):
    L = pk._lib
    ok = pk.CacheDesc(16, 16, 2, 64, 0, 0)
    need = pk.tree_decode_workspace_size(ok)

    def call(desc=ok, out=FAKE, odt=0, q=FAKE, S=1, N=4, H=8, k=FAKE, v=FAKE, bt=FAKE, mb=2,
             ctx=FAKE, start=FAKE, mask=FAKE, words=1, scale=0.1, ws=FAKE, nb=need):
        return L.pa_tree_decode(out, odt, q, S, N, H, k, v, ctypes.byref(desc), bt, mb, ctx, start,
                                mask, words, scale, ws, nb, None, None)
    D = pk.CacheDesc
    for desc in (D(16, 16, 2, 96, 0, 0), D(16, 64, 2, 64, 0, 0), D(16, 16, 2, 64, 2, 0),
                 D(16, 16, 3, 64, 0, 0), D(16, 16, 2, 64, 3, 2)):
        assert call(desc) == pk.PA_ERR_UNSUPPORTED
    assert call(H=2 * 129) == pk.PA_ERR_UNSUPPORTED
    assert call(S=65536) == pk.PA_ERR_UNSUPPORTED
    for bad in (dict(S=-1), dict(N=-1), dict(H=0), dict(mb=-1), dict(odt=3), dict(words=0),
                dict(words=33), dict(scale=float("nan")), dict(out=None), dict(q=None),
                dict(k=None), dict(v=None), dict(bt=None), dict(ctx=None), dict(start=None),
                dict(mask=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(ws=ODD)):
        assert call(**bad) == pk.PA_ERR_INVALID_ARG, bad
        assert L.pa_last_error()
    assert call(ws=None) == pk.PA_ERR_WORKSPACE
    assert call(nb=need - 1) == pk.PA_ERR_WORKSPACE
    assert call(S=0, out=None) == pk.PA_OK
    assert call(N=0, out=None) == pk.PA_OK
    with pytest.raises(ValueError):
        pk.tree_decode_workspace_size(D(16, 16, 2, 96, 0, 0))


def test_compact_refusals(pk):
    L = pk._lib
    ok = pk.CacheDesc(16, 16, 2, 64, 0, 0)
    one = (ctypes.c_void_p * 1)(0x1000)

    def call(k=one, v=one, layers=1, desc=ok, bt=FAKE, mb=2, ctx=FAKE, acc=FAKE, lens=FAKE, S=1,
             path=4):
        return L.pa_tree_compact(k, v, layers, ctypes.byref(desc), bt, mb, ctx, acc, lens, S, path,
                                 None, None)
    assert call(desc=pk.CacheDesc(16, 16, 2, 96, 0, 0)) == pk.PA_ERR_UNSUPPORTED
    assert call(S=65536) == pk.PA_ERR_UNSUPPORTED
    odd = (ctypes.c_void_p * 1)(0x1004)
    null = (ctypes.c_void_p * 1)(None)
    for bad in (dict(layers=0), dict(layers=257), dict(S=-1), dict(path=0), dict(path=1025),
                dict(mb=-1), dict(k=None), dict(v=None), dict(bt=None), dict(ctx=None),
                dict(acc=None), dict(lens=None), dict(k=odd), dict(v=odd), dict(k=null)):
        assert call(**bad) == pk.PA_ERR_INVALID_ARG, bad
    assert call(S=0, k=None, v=None) == pk.PA_OK


def test_binding_refuses_tensors_off_the_gpu(pk):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        pk.tree_mask(i32(4, 1), i32(4), i32(4), i32(2))
    with pytest.raises(ValueError):
        pk.tree_accept(i32(1, 4), i32(1), torch.zeros(1, dtype=torch.int64), i32(4), i32(2),
                       torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int64))
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    q = torch.zeros(4, 8, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        pk.tree_decode(torch.empty_like(q), q, kc, kc, i32(1, 2), i32(1), i32(2), i32(4, 1), 0.1)
    with pytest.raises(ValueError):
        pk.tree_compact([kc], [kc], i32(1, 2), i32(1), i32(1, 4), i32(1))
    with pytest.raises(ValueError):
        pk.tree_compact([], [], i32(1, 2), i32(1), i32(1, 4), i32(1))


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")
def test_calls_without_a_gpu_fail_cleanly(pk):
    L = pk._lib
    for dt in (0, 1, 3):
        desc = pk.CacheDesc(16, 16, 2, 128, dt, 0)
        st = L.pa_tree_decode(FAKE, 0, FAKE, 1, 4, 8, FAKE, FAKE, ctypes.byref(desc), FAKE, 2, FAKE,
                              FAKE, FAKE, 1, 0.1, FAKE, 1 << 40, None, None)
        assert st == pk.PA_ERR_CUDA
    assert L.pa_tree_mask(FAKE, FAKE, FAKE, FAKE, 1, 4, 1, None, None) == pk.PA_ERR_CUDA


# --- the block manager ---------------------------------------------------------------------------

def test_prepare_tree_and_truncate(pk):
    from paged_kv_cache_417_b200.block_manager import BlockManager
    bm = BlockManager(12, 4, [7, 3, 0, 9, 1, 2, 4, 5, 6, 8, 10, 11])
    bm.add_sequence(1)
    bm.add_sequence(2)
    bm.allocate_tokens(1, 6)   # blocks 7, 3
    step = bm.prepare_tree([2, 1], [0, 5], 4)
    assert step["context_lens"].tolist() == [0, 6]
    assert step["tree_start"].tolist() == [0, 0, 5]
    assert step["block_tables"].tolist() == [[-1] * 4, [7, 3, 0, -1]]
    assert step["slot_mapping"].tolist() == [3 * 4 + 2, 3 * 4 + 3, 0, 1, 2]
    assert step["copy_pairs"].shape == (0, 2)
    assert bm.num_tokens(1) == 11 and bm.num_free == 9
    bm.truncate(1, 8)
    assert bm.block_table(1) == [7, 3] and bm.num_free == 10 and bm.ref_count(0) == 0
    bm.truncate(1, 8)
    bm.truncate(1, 5)
    assert bm.block_table(1) == [7, 3] and bm.num_tokens(1) == 5
    bm.truncate(1, 0)
    assert bm.block_table(1) == [] and bm.num_free == 12


def test_prepare_tree_copies_a_shared_last_block_once(pk):
    from paged_kv_cache_417_b200.block_manager import BlockManager
    bm = BlockManager(10, 4)
    bm.add_sequence(1)
    bm.allocate_tokens(1, 6)   # 0, 1
    bm.fork(1, 2)
    step = bm.prepare_tree([1, 2], [3, 1], 4)
    # The first to write copies; the other then holds the block alone.
    assert step["copy_pairs"].tolist() == [[1, 2]]
    assert step["block_tables"].tolist() == [[0, 2, 3, -1], [0, 1, -1, -1]]
    assert step["slot_mapping"].tolist() == [10, 11, 12, 6]
    assert [bm.ref_count(b) for b in range(4)] == [2, 1, 1, 1]
    # An empty tree copies nothing.
    bm.fork(2, 3)
    step = bm.prepare_tree([2], [0], 4)
    assert step["copy_pairs"].shape == (0, 2) and bm.ref_count(1) == 2
    # Truncating a sharer leaves the other its block.
    bm.truncate(3, 4)
    assert bm.ref_count(1) == 1 and bm.block_table(3) == [0]


def test_prepare_tree_refuses_without_change(pk):
    from paged_kv_cache_417_b200.block_manager import BlockManager
    bm = BlockManager(4, 4)
    bm.add_sequence(1)
    bm.add_sequence(2)
    bm.allocate_tokens(1, 5)
    def state():
        return bm.num_free, bm.num_tokens(1), bm.num_tokens(2), bm.block_table(1), bm.block_table(2)
    before = state()
    for seqs, sizes, width in (([1, 2], [4, 9], 4), ([1], [-1], 4), ([1, 1], [1, 1], 4),
                               ([5], [1], 4), ([1], [8], 3), ([1], [2 ** 31 - 1], 4),
                               ([1], [1], 1), ([1], [1], 0), ([1, 2], [2 ** 31 - 1] * 2, 2 ** 20)):
        with pytest.raises(pk.PagedKVError):
            bm.prepare_tree(seqs, sizes, width)
        assert state() == before, (seqs, sizes)
    with pytest.raises(ValueError):
        bm.prepare_tree([1, 2], [1], 4)
    for n in (-1, 6):
        with pytest.raises(pk.PagedKVError):
            bm.truncate(1, n)
    with pytest.raises(pk.PagedKVError):
        bm.truncate(7, 0)
    assert state() == before
    L = pk._lib
    assert L.pa_bm_truncate(None, 1, 0) == pk.PA_ERR_INVALID_ARG
    assert L.pa_bm_prepare_tree(None, None, 0, None, 1, None, None, None, None, None,
                                None) == pk.PA_ERR_INVALID_ARG
    assert bm.prepare_tree([], [], 1)["tree_start"].tolist() == [0]


def test_prepare_tree_refused_for_room_takes_no_memory(pk):
    """A tree far beyond the pool is refused before its table gets any room."""
    L = pk._lib
    from paged_kv_cache_417_b200.block_manager import BlockManager

    def mapped():
        with open("/proc/self/statm") as f:
            return int(f.read().split()[0]) * resource.getpagesize()
    bm = BlockManager(4, 1)
    bm.add_sequence(1)
    seqs, sizes = np.array([1], dtype=np.int64), np.array([2 ** 29], dtype=np.int32)
    room = [np.zeros(2, dtype=np.int64) for _ in range(5)]
    before = mapped()
    st = L.pa_bm_prepare_tree(bm._h, seqs.ctypes.data, 1, sizes.ctypes.data, 2 ** 30,
                              *(x.ctypes.data for x in room), None)
    assert st == pk.PA_ERR_INVALID_ARG and b"pool exhausted" in L.pa_last_error()
    assert mapped() - before < 2 ** 28
    assert bm.num_tokens(1) == 0 and bm.num_free == 4


# --- the plain forms themselves ------------------------------------------------------------------

def test_plain_forms_by_hand():
    par = [-1, 0, 0, 1, 2, 2]
    assert ancestors(par).astype(int).tolist() == [
        [1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 0, 1, 0, 0, 0], [1, 1, 0, 1, 0, 0],
        [1, 0, 1, 0, 1, 0], [1, 0, 1, 0, 0, 1]]
    assert pack_bits(ancestors(par), 1).ravel().tolist() == [1, 3, 5, 11, 21, 37]
    # 5 and 4 hold the same token: the lower one is taken.
    assert accept_path(par, [9, 1, 2, 3, 4, 4], [2, 0, 4, 0, 8, 7], 9) == ([0, 2, 4], 8)
    assert accept_path(par, [9, 1, 2, 3, 4, 4], [2, 0, 4, 0, 8, 7], 2) == ([0, 2], 4)
    assert accept_path([], [], [], 3) == ([], -1)


def test_expected_attention_by_hand():
    """One cached token and a two-node chain with keys that score alike."""
    b = TreeBatch(0, [1], [2], kv_heads=1, group=1, dim=64, shape="chain")
    b.query.zero_()
    out, room = b.expected()
    blk = int(b.table[0, 0])
    v = b.pools[1][blk, 0].double()
    assert torch.allclose(out[0, 0], (v[0] + v[1]) / 2)
    assert torch.allclose(out[1, 0], (v[0] + v[1] + v[2]) / 3)
    assert (room > 0).all() and (room < 0.02).all()
