"""Inputs of drafted-tree steps, and what they should give, in 64 bits and
plain loops: the expected results of the tree tests."""
from __future__ import annotations

import numpy as np
import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def random_parents(rng, n, shape="bushy"):
    """Parents of an n-node tree: a chain, a star, or one random node each."""
    if shape == "chain":
        return [i - 1 for i in range(n)]
    if shape == "star":
        return [-1 if i == 0 else 0 for i in range(n)]
    return [-1 if i == 0 else int(rng.integers(0, i)) for i in range(n)]


def ancestors(parents):
    """[n][n] truth values: node j is node i or an ancestor of it."""
    n = len(parents)
    a = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            a[i] = a[p]
        a[i, i] = True
    return a


def pack_bits(rows, words):
    """int32 [n, words] of truth values [n, m]; columns past 32 * words are
    dropped."""
    out = np.zeros((len(rows), words), dtype=np.uint32)
    for i, r in enumerate(rows):
        for j in np.nonzero(r)[0]:
            if j < 32 * words:
                out[i, j // 32] |= np.uint32(1 << (j % 32))
    return out.view(np.int32)


def accept_path(parents, draft, target, max_path):
    """(path, token after it) by walking the tree."""
    if not parents:
        return [], -1
    path = [0]
    while len(path) < max_path:
        at = path[-1]
        nxt = [c for c in range(len(parents)) if parents[c] == at and draft[c] == target[at]]
        if not nxt:
            break
        path.append(nxt[0])
    return path, target[path[-1]]


def fp8_bytes(values, block_size):
    """fp8 tiles [blocks, heads, bytes] of float values [blocks, heads,
    block_size, dim], as write_kv lays them out."""
    v = values.float()
    amax = v.abs().amax(-1)
    inv = torch.where(amax > 0, 448.0 / amax, torch.zeros_like(amax))
    codes = (v * inv[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = (amax / 448.0).contiguous().view(torch.uint8)
    return torch.cat([codes.flatten(2), scale.flatten(2)], -1).contiguous()


def fp8_values(data, block_size, dim):
    """What the bytes stand for, float64 [blocks, heads, block_size, dim]."""
    n = block_size * dim
    codes = data[..., :n].contiguous().view(torch.float8_e4m3fn).double()
    scale = data[..., n:].contiguous().view(torch.float32).double()
    return codes.reshape(*data.shape[:2], block_size, dim) * scale[..., None]


class TreeBatch:
    """A batch of trees over a scattered paged cache, on the CPU. Slots that
    hold no token are NaN, in used blocks too."""

    def __init__(self, seed, ctx, trees, kv_heads=2, group=4, dim=64, block=16, cache="f16",
                 io=None, masks="tree", shape="bushy", pad=0, lead=0, spare_blocks=3, q_gain=1.0,
                 words=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.rng, self.ctx, self.trees = rng, list(ctx), list(trees)
        self.kv_heads, self.group, self.dim, self.block = kv_heads, group, dim, block
        self.cache, self.io = cache, TYPES[io or ("f16" if cache == "fp8" else cache)]
        self.heads = kv_heads * group
        S = len(self.ctx)
        need = [-(-(c + t) // block) for c, t in zip(self.ctx, self.trees)]
        self.num_blocks = sum(need) + spare_blocks
        ids = rng.permutation(self.num_blocks).tolist()
        width = max(need + [1])
        table = np.full((S, width), -1, dtype=np.int32)
        for s, k in enumerate(need):
            table[s, :k] = ids[:k]
            ids = ids[k:]
        self.table = torch.from_numpy(table)
        filled = torch.zeros(self.num_blocks, block, dtype=torch.bool)
        for s in range(S):
            for j in range(self.ctx[s] + self.trees[s]):
                filled[table[s, j // block], j % block] = True
        shape4 = (self.num_blocks, kv_heads, block, dim)
        self.pools = []
        for _ in range(2):
            x = torch.randn(shape4, generator=g)
            if cache == "fp8":
                data = fp8_bytes(x.to(self.io), block)
                n = block * dim
                codes = data[..., :n].reshape(shape4)
                codes[~filled[:, None].expand(shape4[:3])] = 0x7F
                scale = data[..., n:].contiguous().view(torch.float32)
                scale[~filled[:, None].expand(shape4[:3])] = float("nan")
                data = torch.cat([codes.flatten(2), scale.view(torch.uint8).flatten(2)], -1)
                self.pools.append(data.contiguous())
            else:
                x[~filled[:, None].expand(shape4[:3])] = float("nan")
                self.pools.append(x.to(TYPES[cache]))
        self.start = torch.tensor([lead] + self.trees).cumsum(0).to(torch.int32)
        self.rows = lead + sum(self.trees) + pad
        self.query = (torch.randn(self.rows, self.heads, dim, generator=g) * q_gain).to(self.io)
        self.words = words or max(1, -(-max(self.trees + [1]) // 32))
        self.parents = torch.full((self.rows,), -5, dtype=torch.int32)
        self.allowed = []
        mask = np.full((self.rows, self.words), -1, dtype=np.int32)
        for s, t in enumerate(self.trees):
            a = int(self.start[s])
            par = random_parents(rng, t, shape)
            self.parents[a:a + t] = torch.tensor(par, dtype=torch.int32)
            if masks == "tree":
                ok = ancestors(par)
            elif masks == "none":
                ok = np.zeros((t, t), dtype=bool)
            else:  # any bits, rows without one among them, bits past the end too
                ok = rng.random((t, 32 * self.words)) < rng.random((t, 1)) * \
                    (rng.random((t, 1)) < 0.7)
            mask[a:a + t] = pack_bits(ok, self.words)
            self.allowed.append(ok[:, :t])
        self.mask = torch.from_numpy(mask)
        self.scale = dim ** -0.5

    def values(self, which):
        if self.cache == "fp8":
            return fp8_values(self.pools[which], self.block, self.dim)
        return self.pools[which].double()

    def expected(self, scale=None):
        """(out, room): float64 [rows, heads, dim], NaN rows of no tree, and
        a bound on each element's error before the output is rounded.

        The bound follows the stated precision. With A = sum_j p_j |v_j|:
        rounding p to the row type (fp16 for fp8 caches) is off by at most
        eps/2 of each term, so eps/2 * A; fp16 weights below 2^-14 lose up to
        2^-25 absolutely, n * 2^-25 * max |v| (for fp8 caches, where p times
        the row's scale over at most twice the largest scale is rounded, max
        |v| is at least half of what a lost weight stands for, and weights
        are 2^8 above p); a score summed in fp32 is off by at most
        (dim + 4) * 2^-24 * sum |q||k| * scale = d, which moves p by 2 d
        relatively; exp2 and the scale factor are good to 2^-20; and n terms
        summed in fp32, where a tensor core may truncate, are off by at most
        n * 2^-23 * A."""
        scale = self.scale if scale is None else scale
        out = torch.full((self.rows, self.heads, self.dim), float("nan"), dtype=torch.float64)
        room = torch.zeros_like(out)
        k_all, v_all = self.values(0), self.values(1)
        weights = torch.float16 if self.cache == "fp8" else self.io
        eps = torch.finfo(weights).eps / 2
        for s, t in enumerate(self.trees):
            a, n, c = int(self.start[s]), self.ctx[s] + t, self.ctx[s]
            if t == 0:
                continue
            blocks = self.table[s, :-(-n // self.block)].long()
            k = k_all[blocks].transpose(0, 1).reshape(self.kv_heads, -1, self.dim)[:, :n]
            v = v_all[blocks].transpose(0, 1).reshape(self.kv_heads, -1, self.dim)[:, :n]
            ok = torch.ones(t, n, dtype=torch.bool)
            ok[:, c:] = torch.from_numpy(self.allowed[s])
            q = self.query[a:a + t].double().transpose(0, 1)
            for h in range(self.heads):
                kh, vh = k[h // self.group], v[h // self.group]
                x = (q[h] @ kh.T * scale).masked_fill(~ok, float("-inf"))
                x = torch.where(ok, x, float("-inf"))
                p = torch.softmax(x, -1)
                p = torch.where(ok.any(-1, keepdim=True), p, torch.zeros_like(p))
                for r in range(t):
                    seen = ok[r]
                    out[a + r, h] = p[r, seen] @ vh[seen]
                    # Elements of a row that holds a NaN elsewhere have the same bound.
                    mag = p[r, seen] @ vh[seen].abs()
                    if seen.any():
                        d = (self.dim + 4) * 2.0 ** -24 * abs(scale) * \
                            (q[h][r].abs() @ kh[seen].abs().T).max()
                        sub = n * 2.0 ** -25 * vh[seen].abs().nan_to_num(0, 0, 0).max() \
                            if weights == torch.float16 else 0.0
                        room[a + r, h] = mag * (eps + 2 * d + 2.0 ** -20 + n * 2.0 ** -23) + sub
        return out, room

    def check(self, got, out_dtype=None, expected=None, scale=None):
        """got: [rows, heads, dim], its rows of no tree still NaN."""
        want, room = expected or self.expected(scale)
        g = got.double().cpu()
        dt = out_dtype or got.dtype
        live = torch.zeros(self.rows, dtype=torch.bool)
        live[int(self.start[0]):int(self.start[-1])] = True
        assert torch.isnan(g[~live]).all(), "a row of no tree was written"
        g, want, room = g[live], want[live], room[live]
        fine = torch.isfinite(want)
        same = torch.isnan(g) == torch.isnan(want)
        assert same.all(), f"NaN where there should be none, or none: {torch.nonzero(~same)[:4]}"
        inf = torch.isinf(want)
        assert torch.equal(g[inf], want[inf])
        # Rounding the output: half a step, and the smallest step near zero.
        tiny = torch.finfo(dt).tiny * torch.finfo(dt).eps
        lim = room + (want.abs() + room) * torch.finfo(dt).eps / 2 + tiny + 1e-30
        off = (g - want).abs()
        bad = fine & (off > lim)
        assert not bad.any(), (f"{int(bad.sum())} elements off, worst "
                               f"{float((off / lim)[fine].max()):.2f} of the bound at "
                               f"{torch.nonzero(bad)[0].tolist()}")

    def cuda(self, pk):
        """The call's tensors on the GPU: (query, key, value, table, ctx, start, mask)."""
        pools = [x.cuda() for x in self.pools]
        if self.cache == "fp8":
            pools = [pk.Fp8Cache(x, self.block, self.dim, self.io) for x in pools]
        return (self.query.cuda(), *pools, self.table.cuda(),
                torch.tensor(self.ctx, dtype=torch.int32).cuda(), self.start.cuda(),
                self.mask.cuda())

    def decode(self, pk, out_dtype=None, scale=None, workspace=None, want_err=0):
        q, k, v, table, ctx, start, mask = self.cuda(pk)
        out = torch.full(q.shape, float("nan"), dtype=out_dtype or q.dtype, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pk.tree_decode(out, q, k, v, table, ctx, start, mask,
                       self.scale if scale is None else scale, workspace=workspace, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == want_err, f"device error bits {int(err.item())}"
        return out
