"""The operators of a drafted-tree step over a paged KV cache, for measurement.

A step of tree speculation drafts a small tree of tokens behind each running
sequence, checks all of them in one pass of the model, and keeps the longest
path that the model agrees with:

  tree_mask     parents of each tree's nodes -> ancestor bits and depths
  tree_decode   attention of every node over its sequence's cached context and
                its own ancestors, through the block table
  tree_accept   the accepted path of each tree from the tokens the model picked
  tree_compact  the accepted nodes' K/V rows moved to the slots that follow the
                context, in every layer

The cases take their shapes from the decode benchmark (16-token blocks, head
dimension 128, 32 query heads over 32 or 8 K/V heads, contexts of 128 to 2048
and of 16384 to 32768 tokens) and from the tests (small heads, blocks of 8 and
32 tokens, fp8 caches); trees have 1 to 256 nodes.
"""
import math

import torch

own = False

NODES = 32          # bits in a word of an ancestor mask
ACCEPT_ROOM = 16    # nodes of a path that a step keeps at most
VOCAB = 32000
NEG = float("-inf")


def listed():
    return [
        # One interactive sequence with a short drafted chain: latency counts.
        dict(name="decode_one_chain", op="tree_decode", seqs=1, ctx_lo=300, ctx_hi=300, tree_lo=5,
             tree_hi=5, kv_heads=2, group=4, head_dim=64, block=16, cache="f16", io="f16",
             shape="chain", pad=0),
        # The benchmark's layer with 8 K/V heads, a 16-node tree behind each of its sequences.
        dict(name="decode_layer_kvh8", op="tree_decode", seqs=96, ctx_lo=128, ctx_hi=2048,
             tree_lo=16, tree_hi=16, kv_heads=8, group=4, head_dim=128, block=16, cache="f16",
             io="f16", shape="bushy", pad=0),
        # As many K/V heads as query heads, ragged trees down to none, a padded batch.
        dict(name="decode_mha_ragged", op="tree_decode", seqs=33, ctx_lo=1, ctx_hi=2047,
             tree_lo=0, tree_hi=13, kv_heads=32, group=1, head_dim=128, block=16, cache="f16",
             io="f16", shape="bushy", pad=7),
        # Long contexts, bf16.
        dict(name="decode_long_bf16", op="tree_decode", seqs=8, ctx_lo=16384, ctx_hi=32768,
             tree_lo=24, tree_hi=32, kv_heads=8, group=4, head_dim=128, block=16, cache="bf16",
             io="bf16", shape="bushy", pad=0),
        # Large trees: the widest row tiles, arithmetic counts beside bandwidth.
        dict(name="decode_large_trees", op="tree_decode", seqs=32, ctx_lo=256, ctx_hi=4096,
             tree_lo=64, tree_hi=64, kv_heads=8, group=4, head_dim=128, block=32, cache="f16",
             io="f16", shape="bushy", pad=0),
        # An fp8 cache with bf16 rows.
        dict(name="decode_fp8_bf16", op="tree_decode", seqs=64, ctx_lo=128, ctx_hi=2048,
             tree_lo=8, tree_hi=15, kv_heads=8, group=4, head_dim=128, block=16, cache="fp8",
             io="bf16", shape="bushy", pad=0),
        # One small tree, and a large batch of large ones.
        dict(name="mask_one", op="tree_mask", seqs=1, tree_lo=8, tree_hi=8, shape="bushy", pad=0),
        dict(name="mask_batch", op="tree_mask", seqs=256, tree_lo=1, tree_hi=255, shape="chain",
             pad=9),
        dict(name="accept_one", op="tree_accept", seqs=1, tree_lo=8, tree_hi=8, shape="bushy",
             pad=0, match=70),
        dict(name="accept_batch", op="tree_accept", seqs=256, tree_lo=1, tree_hi=255,
             shape="bushy", pad=9, match=90),
        # A batch whose accepted rows move in all 32 layers, and one layer of one sequence.
        dict(name="compact_layers", op="tree_compact", seqs=64, ctx_lo=8, ctx_hi=96, tree_lo=16,
             tree_hi=16, kv_heads=8, head_dim=128, block=16, cache="f16", layers=32, keep=5),
        dict(name="compact_one", op="tree_compact", seqs=1, ctx_lo=301, ctx_hi=301, tree_lo=7,
             tree_hi=7, kv_heads=4, head_dim=64, block=8, cache="bf16", layers=1, keep=3),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree_decode"] * 5 + ["tree_mask", "tree_accept", "tree_compact"])
    shape = rng.choice(["bushy", "bushy", "chain"])
    if op in ("tree_mask", "tree_accept"):
        hi = _log_int(rng, 1, 256)
        c = dict(op=op, seqs=_log_int(rng, 1, 256), tree_lo=rng.randint(0, hi), tree_hi=hi,
                 shape=shape, pad=rng.choice([0, rng.randint(1, 20)]))
        return dict(c, match=rng.randint(20, 99)) if op == "tree_accept" else c
    if op == "tree_compact":
        hi = _log_int(rng, 2, 64)
        c = dict(op=op, ctx_lo=rng.randint(0, 64), tree_lo=rng.randint(1, hi), tree_hi=hi,
                 kv_heads=rng.choice([1, 2, 4, 5, 8]), head_dim=rng.choice([64, 128]),
                 block=rng.choice([8, 16, 32]), cache=rng.choice(["f16", "bf16"]),
                 layers=_log_int(rng, 1, 32), keep=rng.randint(2, 8))
        # As much in the pools as the largest listed case holds, at most.
        room = 64 * 128 * 8 * 128 * 32 // ((c["ctx_lo"] + 32 + hi + c["block"]) * c["kv_heads"] *
                                           c["head_dim"] * c["layers"])
        return dict(c, ctx_hi=c["ctx_lo"] + rng.randint(0, 32),
                    seqs=_log_int(rng, 1, max(1, min(64, room))))
    cache = rng.choice(["f16", "bf16", "fp8"])
    io = cache if cache != "fp8" else rng.choice(["f16", "bf16"])
    kv, group = rng.choice([(1, 8), (2, 4), (8, 4), (32, 1), (8, 8), (5, 7), (4, 2), (2, 16),
                            (8, 5), (16, 2), (1, 33)])
    tree_hi = _log_int(rng, 1, 128)
    ctx_hi = _log_int(rng, 8, 32768)
    ctx_lo = rng.choice([0, ctx_hi // 2, ctx_hi, rng.randint(0, ctx_hi)])
    # No more cached rows, scores or query rows than the largest listed cases have.
    room = min(2_000_000 // ((ctx_hi + tree_hi) * kv),
               270_000_000 // ((ctx_hi + tree_hi + 32) * tree_hi * kv * group))
    return dict(op=op, seqs=_log_int(rng, 1, max(1, min(96, room))), ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                tree_lo=rng.choice([tree_hi, rng.randint(0, tree_hi)]), tree_hi=tree_hi,
                kv_heads=kv, group=group, head_dim=rng.choice([64, 128]),
                block=rng.choice([8, 16, 32]), cache=cache, io=io, shape=shape,
                pad=rng.choice([0, 0, rng.randint(1, 9)]))


# --- sizes that follow from a case alone ---------------------------------------------------------

def _spread(n, lo, hi, phase):
    """n integers that fill [lo, hi] evenly, in a scattered order."""
    return [lo + int((phase + 0.6180339887498949 * i) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _trees(c):
    t = _spread(c["seqs"], c["tree_lo"], c["tree_hi"], 0.5)
    return [c["tree_hi"]] + t[1:]


def _contexts(c):
    t = _spread(c["seqs"], c["ctx_lo"], c["ctx_hi"], 0.25)
    return t[:-1] + [c["ctx_hi"]]


def _words(c):
    return (c["tree_hi"] + NODES - 1) // NODES


def _row_bytes(c):
    return c["head_dim"] + 4 if c["cache"] == "fp8" else 2 * c["head_dim"]


def _kept(c):
    return [min(c["keep"], t) for t in _trees(c)]


def work(case):
    c, trees = case, _trees(case)
    nodes = sum(trees)
    if c["op"] == "tree_mask":
        return {"bytes": 4 * (nodes * (2 + _words(c)) + c["seqs"] + 1), "flops": nodes}
    if c["op"] == "tree_accept":
        return {"bytes": nodes * (4 + 8 + 8) + 4 * (c["seqs"] + 1) +
                c["seqs"] * (4 * ACCEPT_ROOM + 4 + 8), "flops": nodes}
    ctx = _contexts(c)
    if c["op"] == "tree_compact":
        moved = sum(max(0, k - 1) for k in _kept(c))  # the root stays where it is
        return {"bytes": moved * c["layers"] * 2 * c["kv_heads"] * _row_bytes(c) * 2 +
                8 * c["seqs"] + 4 * c["seqs"] * ACCEPT_ROOM, "flops": 0}
    heads = c["kv_heads"] * c["group"]
    tokens = sum(n + t for n, t in zip(ctx, trees) if t)
    pairs = sum(t * (n + t) for n, t in zip(ctx, trees))
    return {"bytes": tokens * c["kv_heads"] * 2 * _row_bytes(c) +
            nodes * heads * c["head_dim"] * 2 * 2 + 4 * nodes * _words(c) +
            4 * (tokens // c["block"] + 2 * c["seqs"]),
            "flops": 4 * pairs * heads * c["head_dim"]}


# --- inputs --------------------------------------------------------------------------------------

def _parents(trees, shape, g):
    """Parents of every node, -1 for roots: a chain, or a tree in which most
    nodes hang near the front."""
    out = []
    for t in trees:
        i = torch.arange(t)
        back = torch.zeros(t, dtype=torch.int64) if shape == "chain" else \
            (torch.rand(t, generator=g).square() * i).long()
        out.append(torch.where(i > 0, i - 1 - torch.minimum(back, i - 1), -1))
    return torch.cat(out).to(torch.int32)


def _ancestors(parents, trees):
    """bool [seqs, t, t] on the CPU: node i's ancestors and itself."""
    n = max(trees + [1])
    anc = torch.zeros(len(trees), n, n, dtype=torch.bool)
    at = 0
    for s, t in enumerate(trees):
        p = parents[at:at + t].tolist()
        for i in range(t):
            if p[i] >= 0:
                anc[s, i] = anc[s, p[i]]
            anc[s, i, i] = True
        at += t
    return anc


def _packed(anc, words):
    """int32 mask words of bool [..., nodes]."""
    pad = torch.zeros(*anc.shape[:-1], words * NODES, dtype=torch.int64, device=anc.device)
    pad[..., :anc.shape[-1]] = anc[..., :words * NODES]
    pad = pad.reshape(*anc.shape[:-1], words, NODES)
    return (pad << torch.arange(NODES, device=anc.device)).sum(-1).to(torch.int32)


_TYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


def _pool(c, blocks, g, dev):
    x = torch.randn(blocks, c["kv_heads"], c["block"], c["head_dim"], generator=g, device=dev,
                    dtype=torch.float16 if c["cache"] == "fp8" else _TYPE[c["cache"]])
    if c["cache"] != "fp8":
        return x
    x = x.float()
    scale = x.abs().amax(-1) / 448.0
    codes = (x / scale[..., None].clamp(min=1e-20)).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([codes.flatten(2), scale.contiguous().view(torch.uint8).flatten(2)], -1)


def _tables(c, lens, g, dev):
    """Block tables over scattered blocks, and how many blocks there are."""
    need = torch.tensor([(n + c["block"] - 1) // c["block"] for n in lens])
    width = max(1, int(need.max()))
    blocks = max(1, int(need.sum()))
    ids = torch.randperm(blocks, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    table[torch.arange(width) < need[:, None]] = ids[:int(need.sum())]
    return table.to(dev), blocks


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator().manual_seed(seed)
    d = torch.Generator(device=dev).manual_seed(seed)
    mix = torch.randperm(c["seqs"], generator=g).tolist()
    trees = [_trees(c)[i] for i in mix]
    starts = torch.tensor([0] + trees).cumsum(0).to(torch.int32)
    nodes = sum(trees)
    s = dict(case=c, start=starts.to(dev), tmax=max(trees + [1]))
    if c["op"] != "tree_compact":
        parents = _parents(trees, c["shape"], g)
    if c["op"] in ("tree_mask", "tree_accept"):
        tail = torch.full((c["pad"],), -1, dtype=torch.int32)
        s["parents"] = torch.cat([parents, tail]).to(dev)
    if c["op"] == "tree_mask":
        s["mask"] = torch.full((nodes + c["pad"], _words(c)), -7, dtype=torch.int32, device=dev)
        s["depth"] = torch.full((nodes + c["pad"],), -7, dtype=torch.int32, device=dev)
    elif c["op"] == "tree_accept":
        draft = torch.randint(VOCAB, (nodes + c["pad"],), generator=g)
        target = torch.randint(VOCAB, (nodes + c["pad"],), generator=g)
        # Where the model agrees with the draft, it picked the token of one of a node's children.
        child = torch.nonzero(parents >= 0).flatten()
        child = child[torch.randperm(len(child), generator=g)]
        child = child[torch.rand(len(child), generator=g) * 100 < c["match"]]
        owner = torch.repeat_interleave(starts[:-1].long(), torch.tensor(trees))
        up = (parents.long() + owner)[child].numpy()
        tn = target.numpy()
        tn[up] = draft.numpy()[child.numpy()]
        s.update(draft=draft.to(dev), target=target.to(dev),
                 accepted=torch.empty(c["seqs"], ACCEPT_ROOM, dtype=torch.int32, device=dev),
                 lens=torch.empty(c["seqs"], dtype=torch.int32, device=dev),
                 next=torch.empty(c["seqs"], dtype=torch.int64, device=dev))
    else:
        ctx = [_contexts(c)[i] for i in mix]
        table, blocks = _tables(c, [n + t for n, t in zip(ctx, trees)], g, dev)
        s.update(table=table, ctx=torch.tensor(ctx, dtype=torch.int32).to(dev))
        if c["op"] == "tree_compact":
            s["pools"] = torch.randn(2 * c["layers"], blocks, c["kv_heads"], c["block"],
                                     c["head_dim"], generator=d, device=dev,
                                     dtype=_TYPE[c["cache"]])
            s["key"], s["value"] = list(s["pools"][0::2]), list(s["pools"][1::2])
            kept = [_kept(c)[i] for i in mix]
            path = torch.full((c["seqs"], ACCEPT_ROOM), -1, dtype=torch.int32)
            for i, (t, k) in enumerate(zip(trees, kept)):
                rest = torch.randperm(t - 1, generator=g)[:k - 1].sort().values + 1 if k else []
                path[i, :k] = torch.cat([torch.zeros(1, dtype=torch.int64), rest])[:k] if k else 0
            s["accepted"] = path.to(dev)
            s["lens"] = torch.tensor(kept, dtype=torch.int32).to(dev)
        else:
            s["key"], s["value"] = _pool(c, blocks, d, dev), _pool(c, blocks, d, dev)
            heads = c["kv_heads"] * c["group"]
            rows = (nodes + c["pad"], heads, c["head_dim"])
            q = torch.randn(rows, generator=d, device=dev) * 1.5
            s["query"] = q.to(_TYPE[c["io"]])
            s["out"] = torch.full(rows, 0.03125, dtype=_TYPE[c["io"]], device=dev)
            words = _words(c)
            mask = torch.zeros(nodes + c["pad"], words, dtype=torch.int32)
            packed = _packed(_ancestors(parents, trees), words)
            inside = torch.arange(packed.shape[1]) < torch.tensor(trees)[:, None]
            mask[:nodes] = packed[inside]
            s["mask"] = mask.to(dev)
            s["scale"] = c["head_dim"] ** -0.5
    return s


# --- the framework's calls -----------------------------------------------------------------------

def _own(s):
    import paged_kv_cache_417_b200 as pk

    c = s["case"]
    if c["op"] == "tree_mask":
        return pk.tree_mask(s["mask"], s["depth"], s["parents"], s["start"])
    if c["op"] == "tree_accept":
        return pk.tree_accept(s["accepted"], s["lens"], s["next"], s["parents"], s["start"],
                              s["draft"], s["target"])
    if c["op"] == "tree_compact":
        pk.tree_compact(s["key"], s["value"], s["table"], s["ctx"], s["accepted"], s["lens"])
        return s["pools"]
    key, value = s["key"], s["value"]
    if c["cache"] == "fp8":
        key, value = (pk.Fp8Cache(x, c["block"], c["head_dim"], _TYPE[c["io"]])
                      for x in (key, value))
    if "workspace" not in s:
        s["workspace"] = pk.alloc_tree_workspace(key)
    return pk.tree_decode(s["out"], s["query"], key, value, s["table"], s["ctx"], s["start"],
                          s["mask"], s["scale"], workspace=s["workspace"])


# --- the plain forms -----------------------------------------------------------------------------

def _in_trees(s):
    """For each padded place (sequence, node): its row, and whether there is one."""
    start = s["start"].long()
    node = torch.arange(s["tmax"], device=start.device)
    return start[:-1, None] + node, node < (start[1:] - start[:-1])[:, None]


def _plain_ancestors(parent, live):
    """bool [seqs, t, t] of parents [seqs, t] (-1: none)."""
    t = parent.shape[1]
    node = torch.arange(t, device=parent.device)
    up = (parent[:, :, None] == node) | (node[:, None] == node)
    up = (up & live[:, :, None]).float()
    for _ in range(max(1, (t - 1).bit_length())):
        up = (up @ up > 0).float()
    return up > 0


def _plain_mask(s):
    rows, live = _in_trees(s)
    at = rows.clamp(max=s["parents"].shape[0] - 1)
    anc = _plain_ancestors(torch.where(live, s["parents"][at].long(), -1), live)
    mask, depth = s["mask"].clone(), s["depth"].clone()
    mask[rows[live]] = _packed(anc, s["mask"].shape[1])[live]
    depth[rows[live]] = (anc.sum(-1) - 1).to(torch.int32)[live]
    return mask, depth


def _plain_accept(s):
    rows, live = _in_trees(s)
    at = rows.clamp(max=s["parents"].shape[0] - 1)
    parent = torch.where(live, s["parents"][at].long(), -1)
    draft, target = s["draft"][at], s["target"][at]
    t = parent.shape[1]
    node = torch.arange(t, device=parent.device)
    wanted = target.gather(1, parent.clamp(min=0))
    agrees = live & (parent >= 0) & (draft == wanted)
    # Of siblings that agree the lowest counts.
    earlier = (parent[:, :, None] == parent[:, None, :]) & agrees[:, None, :] & \
        (node[None, :] < node[:, None])
    agrees &= ~earlier.any(-1)
    agrees |= live & (node == 0)
    anc = _plain_ancestors(parent, live)
    taken = live & (~anc | agrees[:, None, :]).all(-1)
    depth = anc.sum(-1) - 1
    taken &= depth < ACCEPT_ROOM
    lens = taken.sum(-1)
    path = torch.full((parent.shape[0], ACCEPT_ROOM + 1), -1, device=parent.device)
    place = torch.where(taken, depth, ACCEPT_ROOM)
    path.scatter_(1, place, node.expand_as(place))
    path = path[:, :ACCEPT_ROOM]
    path = torch.where(torch.arange(ACCEPT_ROOM, device=path.device) < lens[:, None], path, -1)
    last = path.gather(1, (lens - 1).clamp(min=0)[:, None])
    after = target.gather(1, last.clamp(min=0))[:, 0]
    return path.to(torch.int32), lens.to(torch.int32), torch.where(lens > 0, after, -1)


def _plain_compact(s):
    block = s["case"]["block"]
    ctx, path = s["ctx"].long()[:, None], s["accepted"].long()
    step = torch.arange(path.shape[1], device=path.device)
    kept = (step < s["lens"][:, None]) & (path >= 0)
    src, dst = (ctx + path.clamp(min=0))[kept], (ctx + step).expand_as(path)[kept]
    seq = torch.arange(path.shape[0], device=path.device)[:, None].expand_as(path)[kept]
    table = s["table"].long()
    rows = s["pools"][:, table[seq, src // block], :, src % block]
    s["pools"][:, table[seq, dst // block], :, dst % block] = rows
    return s["pools"]


def _dense(c, pool, table):
    """The blocks that the tables name as fp32 [seqs, kv_heads, tokens, head_dim]."""
    x = pool[table.clamp(min=0).long()]
    if c["cache"] == "fp8":
        n = c["block"] * c["head_dim"]
        codes = x[..., :n].contiguous().view(torch.float8_e4m3fn).float()
        scale = x[..., n:].contiguous().view(torch.float32)
        x = codes.unflatten(-1, (c["block"], c["head_dim"])) * scale[..., None]
    return x.float().transpose(1, 2).flatten(2, 3)


def _plain_decode(s):
    c = s["case"]
    rows, live = _in_trees(s)
    at = rows.clamp(max=s["query"].shape[0] - 1)
    seqs, t = rows.shape
    key, value = _dense(c, s["key"], s["table"]), _dense(c, s["value"], s["table"])
    n = key.shape[2]
    q = s["query"][at].float().reshape(seqs, t, c["kv_heads"], c["group"], c["head_dim"])
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)
    token = torch.arange(n, device=q.device)
    ctx = s["ctx"].long()[:, None]
    size = live.sum(-1)[:, None]
    node = token - ctx  # [seqs, n]: the tree's nodes lie behind the context
    word = s["mask"][at].long()
    word = word.gather(2, (node.clamp(min=0) // NODES).clamp(max=word.shape[2] - 1)[:, None, :]
                       .expand(seqs, t, n))
    bit = (word >> (node.clamp(min=0) % NODES)[:, None, :]) & 1
    seen = (node < 0)[:, None, :] | ((node < size)[:, None, :] & (bit == 1))
    seen = seen[:, None, :, None, :].expand(seqs, 1, t, c["group"], n).reshape(
        seqs, 1, t * c["group"], n)
    score = torch.where(seen, q @ key.transpose(2, 3) * s["scale"], NEG)
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(top == NEG, 0.0, top)), 0.0)
    del score
    value = torch.where((token < ctx + size)[:, None, :, None], value, 0.0)
    total = p.sum(-1, keepdim=True)
    o = (p @ value) / torch.where(total == 0, 1.0, total)
    o = o.unflatten(2, (t, c["group"])).permute(0, 2, 1, 3, 4).flatten(2, 3)
    out = s["out"].clone()
    out[rows[live]] = o[live].to(out.dtype)
    return out


def run(state):
    if own:
        return _own(state)
    return {"tree_mask": _plain_mask, "tree_accept": _plain_accept, "tree_compact": _plain_compact,
            "tree_decode": _plain_decode}[state["case"]["op"]](state)


# --- the definitions in 64 bits ------------------------------------------------------------------

def _exact_decode(s):
    c = s["case"]
    bs, dim, group = c["block"], c["head_dim"], c["group"]
    out = s["out"].double()
    start, ctx = s["start"].tolist(), s["ctx"].tolist()
    words = s["mask"].cpu().numpy().astype("uint32")

    def cached(pool, blocks, n):
        x = pool[blocks]
        if c["cache"] == "fp8":
            codes = x[..., :bs * dim].reshape(-1, c["kv_heads"], bs, dim)
            x = codes.contiguous().view(torch.float8_e4m3fn).double() * \
                x[..., bs * dim:].contiguous().view(torch.float32).double().unsqueeze(-1)
        return x.double().movedim(1, 0).reshape(c["kv_heads"], -1, dim)[:, :n]

    for i in range(c["seqs"]):
        a, b = start[i], start[i + 1]
        t = b - a
        if t == 0:
            continue
        n = ctx[i] + t
        blocks = s["table"][i, :(n + bs - 1) // bs].long()
        k, v = cached(s["key"], blocks, n), cached(s["value"], blocks, n)
        allow = torch.ones(t, n, dtype=torch.bool)
        for r in range(t):
            for j in range(t):
                allow[r, ctx[i] + j] = bool((int(words[a + r, j // NODES]) >> (j % NODES)) & 1)
        allow = allow.to(out.device)
        q = s["query"][a:b].double()
        for h in range(c["kv_heads"]):
            for u in range(group):
                x = q[:, h * group + u] @ k[h].T * s["scale"]
                x = x.masked_fill(~allow, NEG)
                w = torch.softmax(x, -1)
                out[a:b, h * group + u] = w @ v[h]
    return out


def _exact_compact(s):
    pools = s["pools"].double()
    bs, table = s["case"]["block"], s["table"].tolist()
    ctx, lens, path = s["ctx"].tolist(), s["lens"].tolist(), s["accepted"].tolist()
    for i, n in enumerate(lens):
        for k in range(1, n):  # paths go up, so a row is read before its slot is written again
            a, b = ctx[i] + path[i][k], ctx[i] + k
            if a != b:
                pools[:, table[i][b // bs], :, b % bs] = pools[:, table[i][a // bs], :, a % bs]
    return pools


def exact(case, seed):
    if case["op"] == "tree_decode":
        # The loop over nodes and heads below takes too long for the largest drawn trees.
        if sum(t * t for t in _trees(case)) > 600_000:
            return None
        return _exact_decode(prepare(case, seed))
    if case["op"] == "tree_compact":
        return _exact_compact(prepare(case, seed))
    return None  # whole numbers: they have to be equal
