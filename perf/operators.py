"""Timed cases of the draft-tree operators: one speculative decode step over the sparse KV cache.

The operators and what they compute (T nodes a tree, G = Hq / Hkv, D = 128):

* ``tree_layout``   parents -> one 64-bit visibility word and the position of every node
* ``qk_norm_rope``  per-head RMS norm of queries and keys with the rotation, and the split of a projection row
* ``tree_attn``     attention of the tree's rows over the resident pool slots and the tree's own keys and values
* ``verify_tree``   which drafted tokens stand, from the target's and the draft's probabilities and given random numbers
* ``commit_path``   the accepted nodes' keys and values into the pages and summaries of every layer

Where ``own`` is true, ``run`` makes the package's calls; where it is false it computes the same with elementary
torch operations.
"""

import math

import numpy as np
import torch

own = False

D, P = 128, 16
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence, 1 + 4 drafts in a chain: the smallest call, made once a step
        {"name": "layout_1x5", "op": "layout", "batch": 1, "tree": 5, "shape": "chain"},
        # a serving batch with the widest trees, ragged
        {"name": "layout_256x64", "op": "layout", "batch": 256, "tree": 64, "shape": "tree"},
        # one sequence's 1 + 4 rows of the 32-head layer: latency
        {"name": "rope_1x5", "op": "rope", "batch": 1, "tokens": 5, "hq": 32, "hkv": 8, "norm": True, "far": 4096, "pad": 0},
        # the 64-head layer's step at batch 16, 1 + 7 rows, far positions, projection rows with a tail behind them
        {"name": "rope_16x8", "op": "rope", "batch": 16, "tokens": 8, "hq": 64, "hkv": 8, "norm": True, "far": 524000, "pad": 64},
        # a prompt's chunk of an odd length through the same operator, without norms
        {"name": "rope_1x16111", "op": "rope", "batch": 1, "tokens": 16111, "hq": 32, "hkv": 8, "norm": False, "far": 131072, "pad": 0},
        # one sequence at 32K with a seven-node tree: few units, the cache split over the SMs
        {"name": "attn_1x7", "op": "attn", "batch": 1, "tree": 7, "hq": 32, "hkv": 8, "slots": 128, "context": 32741, "shape": "tree", "free": 0.0},
        # the 64-head 32K layer at batch 16 with 1 + 7 nodes and a tenth of the slots lost: the framework's decode step
        {"name": "attn_16x8", "op": "attn", "batch": 16, "tree": 8, "hq": 64, "hkv": 8, "slots": 128, "context": 32768, "shape": "chain", "free": 0.1},
        # the same layer with the widest trees: 512 query rows a KV head
        {"name": "attn_16x64", "op": "attn", "batch": 16, "tree": 64, "hq": 64, "hkv": 8, "slots": 128, "context": 32768, "shape": "tree", "free": 0.0},
        # one sequence, a chain, the smaller vocabulary: latency
        {"name": "verify_1x5", "op": "verify", "batch": 1, "tree": 5, "vocab": 32000, "shape": "chain", "draft": True, "pad": 0},
        # a batch of trees over a large odd vocabulary (rows that start off a 16-byte boundary)
        {"name": "verify_32x26", "op": "verify", "batch": 32, "tree": 26, "vocab": 151669, "shape": "tree", "draft": True, "pad": 0},
        # one layer, one sequence: latency
        {"name": "commit_1x1", "op": "commit", "layers": 1, "batch": 1, "tree": 5, "hkv": 8, "slots": 32, "blocks": 40},
        # the rows of a 64-layer stack
        {"name": "commit_64x4", "op": "commit", "layers": 64, "batch": 4, "tree": 8, "hkv": 8, "slots": 16, "blocks": 24},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layout", "rope", "rope", "attn", "attn", "attn", "verify", "verify", "commit"])
    shape = rng.choice(["chain", "tree", "tree"])
    if op == "layout":
        return {"op": op, "batch": _log(rng, 1, 256), "tree": _log(rng, 1, 64), "shape": shape}
    if op == "rope":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 3, 4, 5, 8])
        batch = _log(rng, 1, 64)
        most = min(16000, 16000 * 48 // ((hq + 2 * hkv) * batch))
        return {"op": op, "batch": batch, "tokens": _log(rng, 1, max(1, most)), "hq": hq, "hkv": hkv,
                "norm": rng.random() < 0.6, "far": _log(rng, 512, 524000), "pad": rng.choice([0, 0, 8, 136])}
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
        slots = _log(rng, 4, 256)
        batch = _log(rng, 1, max(1, min(32, 16 * 128 // slots)))
        return {"op": op, "batch": batch, "tree": _log(rng, 1, 64), "hq": hq, "hkv": hkv, "slots": slots,
                "context": _log(rng, slots * P + 1, 40000), "shape": shape, "free": rng.choice([0.0, 0.0, 0.1, 0.5])}
    if op == "verify":
        vocab = _log(rng, 1000, 151600)
        tree = _log(rng, 1, 64)
        most = max(1, min(32, 32 * 26 * 151600 // (vocab * tree)))
        return {"op": op, "batch": _log(rng, 1, most), "tree": tree, "vocab": vocab, "shape": shape,
                "draft": rng.random() < 0.7, "pad": rng.choice([0, 0, 3, 64])}
    blocks, tree = _log(rng, 8, 24), _log(rng, 1, 64)
    return {"op": op, "layers": _log(rng, 1, min(64, 64 * 8 // tree)), "batch": _log(rng, 1, 4), "tree": tree, "hkv": rng.choice([1, 2, 8]),
            "slots": max(1, blocks // rng.choice([1, 2, 3])), "blocks": blocks}


# ----------------------------------------------------------------------------------------------- inputs

def _parents(case, g):
    """parent [B][T] and n_nodes [B] int32 (CPU): a chain, or every node under one of the few before it."""
    B, T = case["batch"], case["tree"]
    j = torch.arange(T).repeat(B, 1)
    if case.get("shape", "chain") == "chain":
        parent = j - 1
    else:
        back = torch.floor(torch.rand(B, T, generator=g) * torch.clamp(j.float(), max=6.0)).long()
        parent = torch.where(j > 0, torch.clamp(j - 1 - back, min=0), -1)
    n = torch.full((B,), T)
    if B > 1:                                                # a ragged batch: one sequence in four has fewer nodes
        short = torch.rand(B, generator=g) < 0.25
        n = torch.where(short, torch.floor(torch.rand(B, generator=g) * (T + 1)).long(), n)
    return parent.int(), n.int()


def _masks(parent, n):
    """Visibility words [B][T] int64 from parents that come before their nodes."""
    B, T = parent.shape
    word = torch.zeros(B, T, dtype=torch.int64)
    for j in range(T):
        up = torch.where(parent[:, j] >= 0, word.gather(1, parent[:, j:j + 1].long().clamp(min=0))[:, 0], 0)
        bit = torch.tensor(1 << j if j < 63 else -(1 << 63), dtype=torch.int64)
        word[:, j] = torch.where(j < n, up | bit, 0)
    return word


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator("cuda").manual_seed(seed + 1)
    return {"case": case, "data": _PREPARE[case["op"]](case, g, gd)}


def _randn(gd, *shape):
    return torch.randn(*shape, generator=gd, device="cuda")


def _prepare_layout(case, g, gd):
    parent, n = _parents(case, g)
    ctx = torch.randint(1, 130000, (case["batch"],), generator=g).int()
    B, T = case["batch"], case["tree"]
    return {"parent": parent.cuda(), "n_nodes": n.cuda(), "ctx_len": ctx.cuda(),
            "mask": torch.empty(B, T, dtype=torch.int64, device="cuda"), "pos": torch.empty(B, T, dtype=torch.int32, device="cuda")}


def _prepare_rope(case, g, gd):
    B, T, hq, hkv = case["batch"], case["tokens"], case["hq"], case["hkv"]
    rows = _randn(gd, B, T, (hq + 2 * hkv) * D + case["pad"])
    rows[..., :4] *= 8.0
    start = torch.randint(0, max(1, case["far"] - T), (B, 1), generator=g)
    inv_freq = 1.0 / (1e6 ** (torch.arange(0, D, 2, dtype=torch.float64) / D))
    bf = dict(dtype=torch.bfloat16, device="cuda")
    w = [(1.0 + 0.1 * torch.randn(D, generator=g)).to(**bf) if case["norm"] else None for _ in range(2)]
    return {"qkv": rows.to(torch.bfloat16)[..., :(hq + 2 * hkv) * D], "wq": w[0], "wk": w[1], "inv_freq": inv_freq.float().cuda(),
            "pos": (start + torch.arange(T)).int().cuda(), "q": torch.empty(B, T, hq, D, **bf),
            "k": torch.empty(B, hkv, T, D, **bf), "v": torch.empty(B, hkv, T, D, **bf)}


def _prepare_attn(case, g, gd):
    B, T, hq, hkv, K, ctx = (case[k] for k in ("batch", "tree", "hq", "hkv", "slots", "context"))
    nb = (ctx + P - 1) // P
    parent, n = _parents(case, g)
    kv = _randn(gd, B, hkv, K, 2, P, D)
    kv[..., :4] *= 8.0
    tree = _randn(gd, 2, B, hkv, T, D)
    tree[..., :4] *= 8.0
    slots = torch.rand(B, hkv, nb, generator=gd, device="cuda").argsort(-1)[..., :K].int()
    slots = torch.where(torch.rand(B, hkv, K, generator=gd, device="cuda") < case["free"], -1, slots)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    tree = tree.to(torch.bfloat16)
    # sequences of one batch differ by up to a block, so that last blocks end inside
    lens = ctx - torch.randint(0, min(P, ctx), (B,), generator=g)
    return {"q": _randn(gd, B, T, hq, D).to(torch.bfloat16), "pool": kv.to(torch.bfloat16), "slot_table": slots.int().contiguous(),
            "ctx_len": lens.int().cuda(), "k_tree": tree[0], "v_tree": tree[1], "mask": _masks(parent, n).cuda(), "scale": D ** -0.5,
            "max_blocks": max(nb, K), "out": torch.empty(B, T, hq, D, **bf), "lse": torch.empty(B, T, hq, device="cuda")}


def _prepare_verify(case, g, gd):
    B, T, V = case["batch"], case["tree"], case["vocab"]
    parent, n = _parents(case, g)
    wide = V + case["pad"]
    probs, drafts = (torch.empty(B, T, wide, device="cuda") for _ in range(2))
    tokens = torch.zeros(B, T, dtype=torch.int64, device="cuda")
    pd = parent.cuda().long().clamp(min=0)
    for b in range(B):
        logits = 3.0 * _randn(gd, T, wide)
        probs[b] = torch.softmax(logits, -1)
        drafts[b] = torch.softmax(logits + 0.7 * _randn(gd, T, wide), -1)
        # node j's token is drawn from its parent's draft row (by the exponential race: one pass, no sums)
        race = torch.empty(T, V, device="cuda").exponential_(generator=gd)
        tokens[b] = (drafts[b, pd[b], :V] / race).argmax(-1)
    out = {"probs": probs[..., :V], "draft_probs": drafts[..., :V] if case["draft"] else None, "tokens": tokens.int(),
           "parent": parent.cuda(), "n_nodes": n.cuda(), "u_accept": torch.rand(B, T, generator=gd, device="cuda"),
           "u_sample": torch.rand(B, generator=gd, device="cuda"), "path": torch.empty(B, T, dtype=torch.int32, device="cuda")}
    for name in ("n_accept", "next_token"):
        out[name] = torch.empty(B, dtype=torch.int32, device="cuda")
    return out


def _prepare_commit(case, g, gd):
    L, B, T, H, K, N = (case[k] for k in ("layers", "batch", "tree", "hkv", "slots", "blocks"))
    parent, n = _parents({**case, "shape": "tree"}, g)
    # the path of a random node of each tree, root first
    path = torch.full((B, T), -1, dtype=torch.int32)
    count = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        j = int(torch.randint(0, max(1, int(n[b])), (1,), generator=g)) if n[b] > 0 else -1
        nodes = []
        while j >= 0:
            nodes.append(j)
            j = int(parent[b, j])
        path[b, :len(nodes)] = torch.tensor(nodes[::-1], dtype=torch.int32)
        count[b] = len(nodes)
    ctx = torch.randint(0, N * P - T + 1, (B,), generator=g).int()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    full = _randn(gd, L, B, H, N, 2, P, D).to(torch.bfloat16)
    host = torch.empty(full.shape, dtype=torch.bfloat16, pin_memory=True)
    host.copy_(full)
    slots = torch.rand(L, B, H, N, generator=gd, device="cuda").argsort(-1)[..., :K].int().contiguous()
    tree = _randn(gd, 2, L, B, H, T, D).to(torch.bfloat16)
    pick = slots.long()[..., None, None, None].expand(-1, -1, -1, -1, 2, P, D)
    return {"host_kv": host, "pool": full.gather(3, pick), "slot_table": slots, "kmin": full[..., 0, :, :].amin(-2),
            "kmax": full[..., 0, :, :].amax(-2), "k_tree": tree[0], "v_tree": tree[1], "path": path.cuda(), "n_accept": count.cuda(),
            "ctx_len": ctx.cuda(), "ctx_len_out": torch.empty(B, dtype=torch.int32, device="cuda")}


_PREPARE = {"layout": _prepare_layout, "rope": _prepare_rope, "attn": _prepare_attn, "verify": _prepare_verify,
            "commit": _prepare_commit}


# ------------------------------------------------------------------------------------------ plain forms

def run(state):
    case, s = state["case"], state["data"]
    return _OWN[case["op"]](case, s, state) if own else _PLAIN[case["op"]](case, s)


def _plain_layout(case, s):
    T = case["tree"]
    j = torch.arange(T, device="cuda")
    up = s["parent"].long()
    seen = (j[:, None] == j).expand(case["batch"], T, T).clone()          # [b][node][whom it sees]
    for _ in range(T.bit_length()):                                       # each pass doubles the ancestors known
        far = torch.where((up >= 0)[..., None], seen.gather(1, up.clamp(min=0)[..., None].expand(-1, -1, T)), False)
        seen |= far
        up = torch.where(up >= 0, up.gather(1, up.clamp(min=0)), -1)
    seen &= (j < s["n_nodes"][:, None])[..., None]
    mask = (seen.long() << j).sum(-1)
    depth = torch.clamp(seen.sum(-1) - 1, min=0)
    return {"mask": mask, "pos": (s["ctx_len"][:, None] + depth).int()}


def _plain_rope(case, s):
    hq, hkv = case["hq"], case["hkv"]
    x = s["qkv"].float().unflatten(-1, (-1, D))
    angle = s["pos"].double()[..., None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]

    def turned(h, w):
        if w is not None:
            h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * w.float()
        a, b = h[..., :D // 2], h[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)

    q, k = turned(x[:, :, :hq], s["wq"]), turned(x[:, :, hq:hq + hkv], s["wk"])
    v = x[:, :, hq + hkv:].to(torch.bfloat16)
    return {"q": q, "k": k.transpose(1, 2).contiguous(), "v": v.transpose(1, 2).contiguous()}


def _plain_attn(case, s):
    B, T, hq, hkv, K = (case[k] for k in ("batch", "tree", "hq", "hkv", "slots"))
    G = hq // hkv
    q = s["q"].float().view(B, T, hkv, G, D).transpose(1, 2).reshape(B, hkv, T * G, D)
    keys = torch.cat([s["pool"][:, :, :, 0].reshape(B, hkv, K * P, D), s["k_tree"]], 2).float()
    vals = torch.cat([s["pool"][:, :, :, 1].reshape(B, hkv, K * P, D), s["v_tree"]], 2).float()
    slot = s["slot_table"][..., None]
    cached = ((slot >= 0) & (slot * P + torch.arange(P, device="cuda") < s["ctx_len"][:, None, None, None])).view(B, hkv, 1, K * P)
    bits = (s["mask"][..., None] >> torch.arange(T, device="cuda") & 1).bool()                    # [B, T, T]
    some = bits.any(-1)[:, None, :, None]
    sees = torch.cat([(cached & some).expand(-1, -1, T, -1), bits[:, None].expand(-1, hkv, -1, -1)], -1)
    sees = sees[:, :, :, None].expand(-1, -1, -1, G, -1).reshape(B, hkv, T * G, -1)
    x = torch.where(sees, torch.matmul(q, keys.transpose(-1, -2)) * s["scale"], float("-inf"))
    m = x.amax(-1, keepdim=True)
    w = torch.where(sees, torch.exp(x - m), 0.0)
    total = w.sum(-1, keepdim=True)
    out = torch.where(total > 0, torch.matmul(w, vals) / total, 0.0)
    lse = torch.where(total > 0, m + total.log(), float("-inf"))
    back = lambda t: t.view(B, hkv, T, G, -1).transpose(1, 2).reshape(B, T, hq, -1)  # noqa: E731
    return {"out": back(out).to(torch.bfloat16), "lse": back(lse)[..., 0].contiguous()}


def _plain_verify(case, s):
    B, T, V = case["batch"], case["tree"], case["vocab"]
    seq = torch.arange(B, device="cuda")
    cur = torch.zeros(B, dtype=torch.int64, device="cuda")
    path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    real = s["n_nodes"] > 0
    path[:, 0] = torch.where(real, 0, -1)
    count = real.int()
    left = s["probs"][:, 0].double()
    total = torch.ones(B, dtype=torch.float64, device="cuda")
    for j in range(1, T):                                                  # a node comes after its parent and its elder siblings
        test = (s["parent"][:, j] == cur) & (j < s["n_nodes"])
        x = s["tokens"][:, j].long()
        p = left[seq, x]
        if s["draft_probs"] is not None:
            d = s["draft_probs"][seq, cur].double()
            ok = test & (p > 0) & (s["u_accept"][:, j].double() * total * d[seq, x] < p)
            rest = torch.clamp(left - total[:, None] * d, min=0.0)
            rest_total = rest.sum(-1)
        else:
            ok = test & (p > 0) & (s["u_accept"][:, j].double() * total < p)
            rest = left.clone()
            rest[seq, x] = 0.0
            rest_total = total - p
        no = test & ~ok
        left = torch.where(ok[:, None], s["probs"][:, j].double(), torch.where(no[:, None], rest, left))
        total = torch.where(ok, 1.0, torch.where(no, rest_total, total))
        cur = torch.where(ok, j, cur)
        path.scatter_(1, torch.where(ok, count, 0).long()[:, None], torch.where(ok, j, path[:, 0]).int()[:, None])
        count = count + ok.int()
    left = torch.where((left.sum(-1) > 0)[:, None], left, s["probs"][seq, cur].double())
    cum = left.cumsum(-1)
    over = cum > s["u_sample"].double()[:, None] * cum[:, -1:]
    index = torch.arange(V, device="cuda")
    last = torch.where(left > 0, index, -1).amax(-1)
    token = torch.where(over.any(-1), torch.where(over, index, V).amin(-1), last)
    return {"path": path, "n_accept": count, "next_token": torch.where(real, token, -1).int()}


def _plain_commit(case, s):
    T = case["tree"]
    i = torch.arange(T, device="cuda")
    b, i = torch.nonzero(i < s["n_accept"][:, None], as_tuple=True)
    node = s["path"][b, i].long()
    at = s["ctx_len"][b].long() + i
    block, t = at // P, at % P
    k, v = s["k_tree"][:, b, :, node], s["v_tree"][:, b, :, node]            # [rows, L, H, D]
    hb, hblock, ht = b.cpu(), block.cpu(), t.cpu()
    s["host_kv"][:, hb, :, hblock, 0, ht] = k.cpu()
    s["host_kv"][:, hb, :, hblock, 1, ht] = v.cpu()
    # a block's summary: of its first row where the path opens it, else running
    opens = torch.zeros(case["batch"], case["blocks"], dtype=torch.bool, device="cuda")
    opens[b[t == 0], block[t == 0]] = True
    fresh = opens[None, :, None, :, None]
    spot = (b * case["blocks"] + block)[:, None, None, None]
    for name, way, none in (("kmin", "amin", float("inf")), ("kmax", "amax", float("-inf"))):
        old = torch.where(fresh, none, s[name].float())
        flat = old.permute(1, 3, 0, 2, 4).flatten(0, 1)
        flat.scatter_reduce_(0, spot.expand(-1, *flat.shape[1:]), k.float(), way)
        s[name].copy_(flat.unflatten(0, (case["batch"], case["blocks"])).permute(2, 0, 3, 1, 4))
    hit = s["slot_table"][:, b] == block[:, None, None]                      # [L, rows, H, K]
    layer, row, head, slot = torch.nonzero(hit, as_tuple=True)
    s["pool"][layer, b[row], head, slot, 0, t[row]] = k[row, layer, head]
    s["pool"][layer, b[row], head, slot, 1, t[row]] = v[row, layer, head]
    s["ctx_len_out"].copy_(s["ctx_len"] + s["n_accept"])
    return {name: s[name] for name in ("host_kv", "pool", "kmin", "kmax", "ctx_len_out")}


_PLAIN = {"layout": _plain_layout, "rope": _plain_rope, "attn": _plain_attn, "verify": _plain_verify, "commit": _plain_commit}


# ------------------------------------------------------------------------------------ the package's calls

def _kept(state, make):
    """What a program keeps from step to step: its dims, workspace and layer table."""
    if "kept" not in state:
        state["kept"] = make()
    return state["kept"]


def _own_layout(case, s, state):
    import lookahead_sparse_kv_b200 as lsk
    d = _kept(state, lambda: lsk.make_dims(case["batch"], 1, 1, 8192, 128, 1, 0))
    lsk.tree_layout(d, case["tree"], s["parent"], s["n_nodes"], s["ctx_len"], s["mask"], s["pos"])
    return {"mask": s["mask"], "pos": s["pos"]}


def _own_rope(case, s, state):
    import lookahead_sparse_kv_b200 as lsk
    d = _kept(state, lambda: lsk.make_dims(case["batch"], case["hq"], case["hkv"], 128, 128, 1, 0))
    lsk.qk_norm_rope(d, case["tokens"], s["qkv"], s["wq"], s["wk"], EPS, s["inv_freq"], s["pos"], s["q"], s["k"], s["v"])
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _own_attn(case, s, state):
    import lookahead_sparse_kv_b200 as lsk

    def make():
        d = lsk.make_dims(case["batch"], case["hq"], case["hkv"], s["max_blocks"], case["slots"], 1, 0)
        return d, torch.zeros(lsk.tree_workspace_bytes(d, case["tree"]), dtype=torch.uint8, device="cuda")

    d, ws = _kept(state, make)
    lsk.tree_attn(d, case["tree"], s["q"], s["pool"], s["slot_table"], s["ctx_len"], s["k_tree"], s["v_tree"], s["mask"], s["scale"],
                  s["out"], s["lse"], ws)
    return {"out": s["out"], "lse": s["lse"]}


def _own_verify(case, s, state):
    import lookahead_sparse_kv_b200 as lsk
    d = _kept(state, lambda: lsk.make_dims(case["batch"], 1, 1, 128, 128, 1, 0))
    lsk.verify_tree(d, case["tree"], s["probs"], s["draft_probs"], s["tokens"], s["parent"], s["n_nodes"], s["u_accept"], s["u_sample"],
                    s["path"], s["n_accept"], s["next_token"])
    return {"path": s["path"], "n_accept": s["n_accept"], "next_token": s["next_token"]}


def _own_commit(case, s, state):
    import lookahead_sparse_kv_b200 as lsk

    def make():
        d = lsk.make_dims(case["batch"], case["hkv"], case["hkv"], case["blocks"], case["slots"], 1, 0)
        return d, lsk.make_cache_layers(d, s["host_kv"], s["kmin"], s["kmax"], s["slot_table"], s["pool"])

    d, layers = _kept(state, make)
    lsk.commit_path(d, case["tree"], layers, s["k_tree"], s["v_tree"], s["path"], s["n_accept"], s["ctx_len"], s["ctx_len_out"])
    return {name: s[name] for name in ("host_kv", "pool", "kmin", "kmax", "ctx_len_out")}


_OWN = {"layout": _own_layout, "rope": _own_rope, "attn": _own_attn, "verify": _own_verify, "commit": _own_commit}


# --------------------------------------------------------------------------------------------- the floor

def work(case):
    op = case["op"]
    if op == "layout":
        n = case["batch"] * case["tree"]
        return {"bytes": 16 * n + 8 * case["batch"], "flops": 2 * n}
    if op == "rope":
        n = case["batch"] * case["tokens"]
        heads = case["hq"] + case["hkv"]
        return {"bytes": n * (2 * 2 * D * (heads + case["hkv"]) + 4), "flops": n * heads * D * (7 if case["norm"] else 3)}
    if op == "attn":
        B, T, hq, hkv = case["batch"], case["tree"], case["hq"], case["hkv"]
        tokens = (1.0 - case["free"]) * min(case["slots"] * P, case["context"])
        cache = B * hkv * (tokens + T) * 2 * D * 2
        return {"bytes": cache + B * T * hq * (4 * D + 4) + 4 * B * hkv * case["slots"] + 8 * B * T, "flops": 4.0 * B * T * hq * D * (tokens + T)}
    if op == "verify":
        # the row that the last token is drawn from (the target's, and the draft's where one of its drafts was turned down)
        rows = 2 if case["draft"] else 1
        return {"bytes": case["batch"] * (4.0 * rows * case["vocab"] + 24 * case["tree"]), "flops": 3.0 * rows * case["batch"] * case["vocab"]}
    rows = case["layers"] * case["batch"] * case["hkv"] * (1 + min(4, case["tree"] / 2))
    return {"bytes": rows * (2 + 2) * 2 * D + 4 * case["layers"] * case["batch"] * case["hkv"] * case["slots"], "flops": 4 * rows * D}


# -------------------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed)["data"])


def _exact_layout(case, s):
    parent, n, ctx = (s[k].cpu().tolist() for k in ("parent", "n_nodes", "ctx_len"))
    mask = np.zeros((case["batch"], case["tree"]), dtype=np.uint64)
    pos = np.zeros((case["batch"], case["tree"]), dtype=np.int32)
    for b in range(case["batch"]):
        for j in range(case["tree"]):
            k, steps, word = j, 0, 0
            while j < n[b] and k >= 0:
                word, steps, k = word | 1 << k, steps + 1, parent[b][k]
            mask[b, j], pos[b, j] = word, ctx[b] + max(0, steps - 1)
    return {"mask": mask.view(np.int64), "pos": pos}


def _exact_rope(case, s):
    hq, hkv, B, T = case["hq"], case["hkv"], case["batch"], case["tokens"]
    f64 = dict(dtype=torch.float64, device="cuda")
    q, k, v = torch.empty(B, T, hq, D, **f64), torch.empty(B, hkv, T, D, **f64), torch.empty(B, hkv, T, D, **f64)
    for b in range(B):
        for t in range(0, T, 4096):
            x = s["qkv"][b, t:t + 4096].double()
            n = x.shape[0]
            x = x.reshape(n, -1, D)
            ring = torch.polar(torch.ones(n, D // 2, **f64), torch.outer(s["pos"][b, t:t + 4096].double(), s["inv_freq"].double()))
            for lo, hi, w in ((0, hq, s["wq"]), (hq, hq + hkv, s["wk"])):
                y = x[:, lo:hi]
                if w is not None:
                    y = y / ((y * y).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
                z = torch.complex(y[..., :D // 2].contiguous(), y[..., D // 2:].contiguous()) * ring[:, None]
                y = torch.cat([z.real, z.imag], -1)
                if lo == 0:
                    q[b, t:t + n] = y
                else:
                    k[b, :, t:t + n] = y.transpose(0, 1)
            v[b, :, t:t + n] = x[:, hq + hkv:].transpose(0, 1)
    return {"q": q, "k": k, "v": v}


def _exact_attn(case, s):
    B, T, hq, hkv, K = (case[k] for k in ("batch", "tree", "hq", "hkv", "slots"))
    G = hq // hkv
    out = torch.zeros(B, T, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, hq), float("-inf"), dtype=torch.float64, device="cuda")
    ctx, table = s["ctx_len"].tolist(), s["slot_table"].cpu()
    word = [[int(m) & 0xFFFFFFFFFFFFFFFF for m in row] for row in s["mask"].tolist()]
    for b in range(B):
        seen = torch.tensor([[word[b][j] >> i & 1 for i in range(T)] for j in range(T)], dtype=torch.bool, device="cuda")
        rows = [j for j in range(T) if word[b][j]]
        if not rows:
            continue
        for h in range(hkv):
            first = table[b, h].long() * P
            keep = ((first[:, None] >= 0) & (first[:, None] + torch.arange(P) < ctx[b])).flatten().cuda()
            kv = s["pool"][b, h].double()
            keys = torch.cat([kv[:, 0].reshape(-1, D)[keep], s["k_tree"][b, h].double()])
            vals = torch.cat([kv[:, 1].reshape(-1, D)[keep], s["v_tree"][b, h].double()])
            y = torch.einsum("tgd,nd->gtn", s["q"][b, rows, h * G:(h + 1) * G].double(), keys) * s["scale"]
            y[:, :, -T:].masked_fill_(~seen[rows], float("-inf"))
            lse[b, rows, h * G:(h + 1) * G] = torch.logsumexp(y, -1).T
            out[b, rows, h * G:(h + 1) * G] = torch.einsum("gtn,nd->tgd", torch.softmax(y, -1), vals)
    return {"out": out, "lse": lse}


def _exact_verify(case, s):
    B, T = case["batch"], case["tree"]
    parent, n, tokens = (s[k].cpu().tolist() for k in ("parent", "n_nodes", "tokens"))
    u, us = s["u_accept"].double().cpu().numpy(), s["u_sample"].double().cpu().numpy()
    path, count, token = np.full((B, T), -1, np.int32), np.zeros(B, np.int32), np.full(B, -1, np.int32)
    for b in range(B):
        if not n[b]:
            continue
        nodes, j = [0], 0
        while True:
            mass = s["probs"][b, j].double().cpu().numpy()
            draft = s["draft_probs"][b, j].double().cpu().numpy() if case["draft"] else None
            size, stands = 1.0, None
            for c in (c for c in range(j + 1, n[b]) if parent[b][c] == j):
                x = tokens[b][c]
                if mass[x] > 0 and u[b, c] * size * (draft[x] if case["draft"] else 1.0) < mass[x]:
                    stands = c
                    break
                if case["draft"]:
                    mass = np.maximum(mass - size * draft, 0.0)
                    size = float(mass.sum())
                else:
                    size -= float(mass[x])
                    mass[x] = 0.0
            if stands is None:
                break
            j = stands
            nodes.append(j)
        if not mass.sum() > 0:
            mass = s["probs"][b, j].double().cpu().numpy()
        steps = np.cumsum(mass)
        at = int(np.searchsorted(steps, us[b] * steps[-1], side="right"))
        token[b] = at if at < len(mass) else int(np.nonzero(mass)[0][-1])
        path[b, :len(nodes)], count[b] = nodes, len(nodes)
    return {"path": path, "n_accept": count, "next_token": token}


def _exact_commit(case, s):
    ctx, count, path = (s[k].cpu().tolist() for k in ("ctx_len", "n_accept", "path"))
    table = s["slot_table"].cpu()
    host, pool, low, high = s["host_kv"], s["pool"], s["kmin"], s["kmax"]
    for b in range(case["batch"]):
        for i in range(count[b]):
            block, t = divmod(ctx[b] + i, P)
            k, v = s["k_tree"][:, b, :, path[b][i]], s["v_tree"][:, b, :, path[b][i]]
            host[:, b, :, block, 0, t], host[:, b, :, block, 1, t] = k.cpu(), v.cpu()
            low[:, b, :, block] = k if t == 0 else torch.minimum(low[:, b, :, block], k)
            high[:, b, :, block] = k if t == 0 else torch.maximum(high[:, b, :, block], k)
            for layer, head, slot in torch.nonzero(table[:, b] == block).tolist():
                pool[layer, b, head, slot, 0, t], pool[layer, b, head, slot, 1, t] = k[layer, head], v[layer, head]
    return {"host_kv": host, "pool": pool, "kmin": low, "kmax": high, "ctx_len_out": torch.tensor([c + n for c, n in zip(ctx, count)], dtype=torch.int32)}


_EXACT = {"layout": _exact_layout, "rope": _exact_rope, "attn": _exact_attn, "verify": _exact_verify, "commit": _exact_commit}
