"""The draft-tree calls on the GPU against their fp64 statements (oracle/tree_oracle.py): sizes and masks where each can go
wrong, then a whole speculative step as a program runs it.

Tolerances.  A bf16 output rounds once: 2^-8 of its value.  On top of that
  * qk_norm_rope computes in fp32: a turned pair sums two products whose sizes may cancel, so the absolute part is taken from the
    pair's length, a few fp32 steps: 2^-8 |y| + 2^-20 len.
  * tree_attn sums fp32 products; its softmax weights enter the second product rounded to bf16, each off by at most half a step:
    bf16 keeps 8 significant bits, torch.finfo(bf16).eps = 2^-7, half a step 2^-8 of the weight.  So the sum over the tokens is off
    by at most 2^-8 sum w |v| = 2^-8 A, and the store rounds once more: 2^-8 |o| + 2^-8 A (and 2^-16 A of the two together),
    A = the weighted mean of |v|.  lse: fp32 scores are off by a few 2^-24 sum |q_c k_c|, bounded here by 1e-4.
"""

import math

import numpy as np
import pytest
import torch

import lookahead_sparse_kv_b200 as lsk
from lookahead_sparse_kv_b200 import workloads as W
from oracle import bf16_bits_to_f64
from oracle import tree_oracle as TO

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from lookahead_sparse_kv_b200 import build
    build.build()
    lsk.lib()
    yield
    assert lsk.read_device_error(clear=True) == 0


def f64(t):
    return bf16_bits_to_f64(W.bf16_bits(t))


def make_tree(B, T, g, shape="tree", ragged=True):
    j = torch.arange(T).repeat(B, 1)
    if shape == "chain":
        parent = j - 1
    elif shape == "star":
        parent = torch.where(j > 0, 0, -1)
    else:
        parent = torch.where(j > 0, (torch.rand(B, T, generator=g) * j).floor().long(), -1)
    n = torch.full((B,), T)
    if ragged and B > 1:
        n = torch.randint(0, T + 1, (B,), generator=g)
        n[0], n[-1] = T, 0
    return parent.int(), n.int()


# ------------------------------------------------------------------------------------------ tree_layout

@pytest.mark.parametrize("B,T,shape", [(1, 1, "tree"), (3, 2, "chain"), (5, 31, "tree"), (2, 32, "chain"), (9, 33, "tree"),
                                       (4, 64, "chain"), (130, 64, "tree"), (2, 64, "star")])
def test_tree_layout_matches(B, T, shape):
    g = torch.Generator().manual_seed(B * 100 + T)
    parent, n = make_tree(B, T, g, shape)
    ctx = torch.randint(0, 500000, (B,), generator=g).int()
    d = lsk.make_dims(B, 8, 2, 64, 16, 1, 0)
    mask, pos = torch.full((B, T), -3, dtype=torch.int64, device=DEV), torch.full((B, T), -3, dtype=I32, device=DEV)
    lsk.tree_layout(d, T, parent.to(DEV), n.to(DEV), ctx.to(DEV), mask, pos)
    m, p = TO.tree_layout(parent.numpy(), n.numpy(), ctx.numpy())
    assert np.array_equal(mask.cpu().numpy().view(np.uint64), m) and np.array_equal(pos.cpu().numpy(), p)
    lsk.tree_layout(d, T, parent.to(DEV), None, ctx.to(DEV), mask, pos)                 # every node real
    m, p = TO.tree_layout(parent.numpy(), np.full(B, T), ctx.numpy())
    assert np.array_equal(mask.cpu().numpy().view(np.uint64), m) and np.array_equal(pos.cpu().numpy(), p)


def test_tree_layout_flags_bad_parents_and_counts():
    d = lsk.make_dims(2, 8, 2, 64, 16, 1, 0)
    parent = torch.tensor([[-1, 0, 2, 1], [-1, -5, 9, 0]], dtype=I32, device=DEV)
    n = torch.tensor([4, 77], dtype=I32, device=DEV)
    ctx = torch.tensor([5, 7], dtype=I32, device=DEV)
    mask, pos = torch.empty(2, 4, dtype=torch.int64, device=DEV), torch.empty(2, 4, dtype=I32, device=DEV)
    lsk.tree_layout(d, 4, parent, n, ctx, mask, pos)
    assert mask.tolist() == [[1, 3, 4, 11], [1, 2, 4, 9]] and pos.tolist() == [[5, 6, 5, 7], [7, 7, 7, 8]]
    assert lsk.read_device_error(clear=True) == lsk.DEVERR_ID_RANGE


# ----------------------------------------------------------------------------------------- qk_norm_rope

@pytest.mark.parametrize("B,T,hq,hkv,norm,pad,far", [
    (1, 1, 1, 1, True, 0, 0), (1, 5, 32, 8, True, 0, 40000), (3, 7, 5, 1, True, 8, 524287), (2, 8, 64, 8, False, 136, 131071),
    (2, 33, 6, 3, "q", 0, 1000), (1, 3001, 8, 2, "k", 64, 521000), (64, 1, 32, 8, True, 0, 17000)])
def test_qk_norm_rope_matches(B, T, hq, hkv, norm, pad, far):
    g = torch.Generator().manual_seed(T)
    heads = hq + 2 * hkv
    rows = torch.randn(B, T, heads * 128 + pad, generator=g)
    rows[..., ::37] *= 20.0
    rows = rows.to(BF).to(DEV)
    qkv = rows[..., :heads * 128]
    wq = (1 + 0.2 * torch.randn(128, generator=g)).to(BF).to(DEV) if norm in (True, "q") else None
    wk = (1 + 0.2 * torch.randn(128, generator=g)).to(BF).to(DEV) if norm in (True, "k") else None
    inv = (5e5 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(DEV)
    pos = (far + torch.randint(0, 100, (B, T), generator=g)).int().to(DEV)
    d = lsk.make_dims(B, hq, hkv, 64, 16, 1, 0)
    q, k, v = (torch.full(s, 7.0, dtype=BF, device=DEV) for s in ((B, T, hq, 128), (B, hkv, T, 128), (B, hkv, T, 128)))
    lsk.qk_norm_rope(d, T, qkv, wq, wk, 1e-6, inv, pos, q, k, v)
    x = f64(qkv).reshape(B, T, heads, 128)
    refs = TO.qk_norm_rope(x, hq, hkv, None if wq is None else f64(wq), None if wk is None else f64(wk), 1e-6, inv.cpu().numpy(),
                           pos.cpu().numpy())
    for got, ref in zip((q, k), refs):
        got = f64(got)
        length = np.hypot(ref[..., :64], ref[..., 64:])
        room = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * np.concatenate([length, length], -1)
        assert bool((np.abs(got - ref) <= room).all())
    assert np.array_equal(f64(v), refs[2])


def test_qk_norm_rope_zero_rows_and_wild_values_stay_in_their_heads():
    """An all-zero head gives zeros (eps keeps the norm finite); NaN and infinities stay in their own head."""
    d = lsk.make_dims(1, 2, 1, 64, 16, 1, 0)
    x = torch.randn(1, 3, 4 * 128, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    x[0, 0, :128] = 0
    x[0, 1, 130] = float("nan")
    x[0, 2, 400] = float("inf")
    w = torch.ones(128, dtype=BF, device=DEV)
    inv, pos = torch.ones(64, device=DEV), torch.zeros(1, 3, dtype=I32, device=DEV)
    q, k, v = (torch.empty(s, dtype=BF, device=DEV) for s in ((1, 3, 2, 128), (1, 1, 3, 128), (1, 1, 3, 128)))
    lsk.qk_norm_rope(d, 3, x, w, w, 1e-6, inv, pos, q, k, v)
    assert (q[0, 0, 0] == 0).all()
    assert q[0, 1, 1].isnan().all() and q.isnan().sum() == 128 and not k.isnan().any()
    assert torch.equal(v[0, 0], x[0, :, 384:])


# -------------------------------------------------------------------------------------------- tree_attn

class Attn:
    """Inputs of one tree_attn call and its comparison."""

    def __init__(self, B, T, hq, hkv, K, N, seed, shape="tree", free=0.2, ctx=None, ragged=True):
        g = self.g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.hq, self.hkv, self.K, self.N = B, T, hq, hkv, K, N
        self.d = lsk.make_dims(B, hq, hkv, N, K, 1, 0)
        self.q = torch.randn(B, T, hq, 128, generator=g).to(BF)
        pool = torch.randn(B, hkv, K, 2, 16, 128, generator=g)
        pool[..., :3] *= 6.0
        self.pool = pool.to(BF)
        self.k, self.v = (torch.randn(B, hkv, T, 128, generator=g).to(BF) for _ in range(2))
        self.ctx = torch.tensor(ctx if ctx is not None else [max(0, N * 16 - 5 - 7 * b) for b in range(B)], dtype=I32)
        st = torch.stack([torch.randperm(N, generator=g)[:K] for _ in range(B * hkv)]).view(B, hkv, K)
        self.st = torch.where(torch.rand(B, hkv, K, generator=g) < free, -1, st).int()
        self.parent, self.n = make_tree(B, T, g, shape, ragged)
        self.mask = torch.from_numpy(TO.tree_layout(self.parent.numpy(), self.n.numpy(), self.ctx.numpy())[0].view(np.int64))
        self.scale = 128 ** -0.5
        self.ws = torch.zeros(lsk.tree_workspace_bytes(self.d, T), dtype=torch.uint8, device=DEV)

    def call(self, ws=None, stream=None):
        out = torch.full((self.B, self.T, self.hq, 128), 9.0, dtype=BF, device=DEV)
        lse = torch.full((self.B, self.T, self.hq), 9.0, device=DEV)
        dev = [t.to(DEV) for t in (self.q, self.pool, self.st, self.ctx, self.k, self.v, self.mask)]
        lsk.tree_attn(self.d, self.T, *dev, self.scale, out, lse, self.ws if ws is None else ws, stream=stream)
        torch.cuda.synchronize()
        return out, lse

    def reference(self):
        pool = f64(self.pool)
        args = (f64(self.q), pool[:, :, :, 0], pool[:, :, :, 1], self.st.numpy(), self.ctx.numpy(), f64(self.k), f64(self.v),
                self.mask.numpy().view(np.uint64), self.scale)
        o, lse = TO.tree_attention(*args)
        size, _ = TO.tree_attention(args[0], args[1], np.abs(args[2]), *args[3:6], np.abs(args[6]), *args[7:])
        return o, lse, size

    def check(self):
        out, lse = self.call()
        o, l, size = self.reference()
        got = f64(out)
        over = np.abs(got - o) - (2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -16) * size + 1e-30)
        assert not bool((over > 0).any()), over.max()
        lse = lse.cpu().double().numpy()
        fin = np.isfinite(l)
        assert np.array_equal(np.isfinite(lse), fin) and (lse[~fin] == -np.inf).all()
        assert np.abs(lse[fin] - l[fin]).max(initial=0.0) <= 1e-4
        return out, lse


@pytest.mark.parametrize("B,T,hq,hkv,K,N,shape", [
    (1, 1, 1, 1, 1, 4, "tree"), (1, 5, 8, 2, 16, 40, "chain"), (3, 7, 4, 1, 9, 30, "tree"), (2, 8, 16, 2, 32, 32, "tree"),
    (2, 13, 10, 2, 20, 64, "tree"), (1, 16, 8, 2, 128, 300, "star"), (2, 17, 6, 2, 24, 64, "tree"), (3, 26, 8, 2, 40, 80, "tree"),
    (2, 33, 3, 1, 16, 40, "tree"), (1, 64, 1, 1, 8, 20, "chain"), (2, 64, 8, 1, 33, 50, "tree"), (1, 64, 16, 2, 128, 200, "chain"),
    (1, 40, 7, 1, 17, 32, "tree"), (1, 9, 64, 1, 12, 20, "tree"), (1, 3, 80, 2, 12, 20, "tree"), (2, 31, 12, 3, 70, 90, "star")])
def test_tree_attn_matches(B, T, hq, hkv, K, N, shape):
    Attn(B, T, hq, hkv, K, N, seed=T * 31 + hq, shape=shape).check()


@pytest.mark.parametrize("T,hq", [(1, 4), (5, 4), (16, 4), (20, 8), (64, 4)])
def test_tree_attn_short_and_empty_caches(T, hq):
    """No context, one token, a block that ends inside, every slot free: the tree alone (and nothing at all) still works."""
    a = Attn(5, T, hq, 2, 12, 20, seed=T, ctx=[0, 1, 17, 320, 100], free=0.0, ragged=False)
    a.st[3] = -1                                   # context, but nothing resident
    a.st[4, 0] = -1                                # one head empty, the other not
    a.mask[4, 0] = 0                               # an empty row among others
    a.check()


@pytest.mark.parametrize("T,hq", [(6, 8), (17, 4), (50, 8), (64, 8)])
def test_tree_attn_any_visibility_words(T, hq):
    """Words that no tree makes: random sets, empty rows, bits at and above T, rows that do not see themselves."""
    a = Attn(3, T, hq, 2, 16, 20, seed=T + 1)
    words = torch.randint(-(1 << 62), 1 << 62, (3, T), generator=a.g) * 2 + torch.randint(0, 2, (3, T), generator=a.g)
    words[torch.rand(3, T, generator=a.g) < 0.3] = 0
    a.mask = words
    first = a.call()
    keep = (1 << T) - 1 if T < 64 else -1
    a.mask = words & keep
    a.check()
    again = a.call()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("T,hq,ctx", [(8, 8, 200), (8, 8, 0), (40, 8, 200), (64, 4, 0), (64, 8, 319)])
def test_tree_attn_wild_values_reach_only_rows_that_see_them(T, hq, ctx):
    """NaN and infinities in padding nodes, in free slots, behind the context and in nodes that some rows do not see."""
    a = Attn(2, T, hq, 2, 12, 20, seed=3, ctx=[ctx, ctx], ragged=False, free=0.3)
    a.n[1] = T - 2
    a.mask = torch.from_numpy(TO.tree_layout(a.parent.numpy(), a.n.numpy(), a.ctx.numpy())[0].view(np.int64))
    clean, _ = a.call()
    o, _, _ = a.reference()
    a.k[1, :, T - 2:], a.v[1, :, T - 2:] = float("nan"), float("inf")              # padding
    for h in range(2):
        for s in range(12):
            nv = max(0, min(16, ctx - int(a.st[1, h, s]) * 16)) if a.st[1, h, s] >= 0 else 0
            a.pool[1, h, s, :, nv:] = float("nan")                                 # free or past the context
    same, lse = a.call()
    assert torch.equal(same, clean) and not lse.isnan().any()
    node = T // 2
    a.v[0, 1, node, 5], a.v[0, 1, node, 6] = float("inf"), float("nan")
    out, lse = a.call()
    assert not lse.isnan().any()
    sees = torch.tensor([int(w) >> node & 1 for w in a.mask[0].tolist()], dtype=torch.bool)
    heads = slice(hq // 2, hq)
    assert sees.any() and not sees.all()
    assert (out[0, sees, heads, 5] == float("inf")).all() and out[0, sees, heads, 6].isnan().all()
    out[0, sees, heads, 5:7] = clean[0, sees, heads, 5:7]
    # the product now holds 0 in the two places, and nothing else moved
    assert torch.equal(out, clean)
    a.k[0, 1, node, 9] = float("nan")                                              # a key: its rows become NaN, the others stay
    out, lse = a.call()
    assert out[0, sees, heads].isnan().all() and not out[0, ~sees].isnan().any() and torch.equal(out[0, ~sees], clean[0, ~sees])


@pytest.mark.parametrize("T,hq,K", [(4, 8, 12), (40, 8, 12), (64, 8, 12), (4, 8, 400)])
def test_tree_attn_scores_of_minus_infinity(T, hq, K):
    """A node's key with an infinity: the rows with a score of -inf there give it no weight, whether or not they see anything else
    (the root's row sees nothing else of the tree), and rows with a score of +inf are NaN."""
    a = Attn(1, T, hq, 2, K, K, seed=13, free=0.0, ragged=False)
    a.k[0, 0, 0, 7] = float("inf")                 # the root, seen by every row
    a.q[:, :, :, 7] = -1.0
    a.q[0, T - 1, 0, 7] = 1.0
    out, lse = a.call()
    o, l, size = a.reference()
    bad = np.zeros(o.shape[:3], bool)
    bad[0, T - 1, 0] = True
    assert out.cpu().float().isnan().all(-1).numpy()[bad].all() and not out.cpu().float().isnan().any(-1).numpy()[~bad].any()
    over = np.abs(f64(out) - o) - (2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -16) * size + 1e-30)
    assert not bool((over[~bad] > 0).any())
    assert np.abs(lse.cpu().double().numpy() - l)[~bad].max() <= 1e-4
    a.st[:] = -1                                   # no cache: the root's row has nothing but a score of -inf
    a.parent[0, 1:] = -1
    a.mask = torch.from_numpy(TO.tree_layout(a.parent.numpy(), a.n.numpy(), a.ctx.numpy())[0].view(np.int64))
    out, lse = a.call()
    assert not out[0, 0, :hq // 2].any() and (lse[0, 0, :hq // 2] == float("-inf")).all()
    assert not out[0, 1:].isnan().any()


def test_tree_attn_far_apart_scores():
    """Scores thousands apart, in both orders along the cache, and a tree that outweighs or vanishes beside it."""
    for sign in (1.0, -1.0):
        a = Attn(1, 6, 8, 2, 64, 64, seed=5, free=0.0, ragged=False)
        a.pool[..., 0, :, :] *= (torch.linspace(1, 40, 64).view(1, 1, 64, 1, 1) if sign > 0 else torch.linspace(40, 1, 64).view(1, 1, 64, 1, 1)).to(BF)
        a.k *= 60.0 if sign > 0 else 0.01
        out, lse = a.call()
        o, l, size = a.reference()
        assert not bool((np.abs(f64(out) - o) > 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -16) * size).any())
        # scores of several hundred carry fp32's own step of the sum: 2^-24 * sum |q k| * scale, here below 2e-3
        assert np.abs(lse.cpu().double().numpy() - l).max() <= 2e-3


@pytest.mark.parametrize("T", [8, 64])
def test_tree_attn_agrees_with_sparse_attn_on_the_cache(T):
    """With the tree's scores out of reach (keys far below), the rows give what sparse_attn gives over the same slots."""
    a = Attn(2, T, 8, 8, 32, 40, seed=11, ragged=False)
    q = a.q[:, :1].expand(-1, T, -1, -1).contiguous()
    a.q = q
    a.k = -40.0 * q.float().mean(1).to(BF).view(2, 8, 1, 128).expand(-1, -1, T, -1).contiguous()
    out, lse = a.call()
    d = lsk.make_dims(2, 8, 8, 40, 32, 1, 0)
    o1, l1 = torch.empty(2, 1, 8, 128, device=DEV), torch.empty(2, 1, 8, device=DEV)
    ws = torch.zeros(lsk.workspace_bytes(d), dtype=torch.uint8, device=DEV)
    lsk.sparse_attn(d, q[:, :1].contiguous().to(DEV), a.pool.to(DEV), a.st.to(DEV), a.ctx.to(DEV), a.scale, o1, l1, ws)
    assert torch.allclose(lse, l1.expand(-1, T, -1), atol=1e-4)
    assert torch.allclose(out.float(), o1.expand(-1, T, -1, -1), atol=2e-2, rtol=1e-2)


# ------------------------------------------------------------------------------------------ verify_tree

def verify_inputs(B, T, V, g, shape="tree", pad=0, noise=0.8, temp=2.0, ragged=True):
    parent, n = make_tree(B, T, g, shape, ragged)
    logits = temp * torch.randn(B, T, V + pad, generator=g)
    probs, draft = torch.softmax(logits, -1), torch.softmax(logits + noise * torch.randn(B, T, V + pad, generator=g), -1)
    race = torch.empty(B, T, V).exponential_(generator=g)
    rows = draft.gather(1, parent.long().clamp(min=0)[..., None].expand(-1, -1, V + pad))[..., :V]
    tokens = (rows / race).argmax(-1).int()
    return probs, draft, tokens, parent, n, torch.rand(B, T, generator=g), torch.rand(B, generator=g)


def run_verify(probs, draft, tokens, parent, n, ua, us, V):
    B, T = tokens.shape
    d = lsk.make_dims(B, 1, 1, 64, 16, 1, 0)
    path, cnt, nxt = (torch.full(s, -9, dtype=I32, device=DEV) for s in ((B, T), (B,), (B,)))
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    p, q = dev(probs)[..., :V], None if draft is None else dev(draft)[..., :V]
    lsk.verify_tree(d, T, p, q, dev(tokens), dev(parent), dev(n), dev(ua), dev(us), path, cnt, nxt)
    return path.cpu().numpy(), cnt.cpu().numpy(), nxt.cpu().numpy()


@pytest.mark.parametrize("B,T,V,shape,draft,pad", [
    (1, 1, 1, "tree", True, 0), (2, 2, 3, "chain", True, 1), (4, 5, 33, "chain", False, 0), (5, 9, 1000, "tree", True, 3),
    (3, 64, 257, "star", True, 0), (3, 64, 257, "star", False, 0), (6, 26, 4099, "tree", True, 5), (6, 26, 4099, "tree", False, 64),
    (2, 8, 50257, "tree", True, 0), (40, 7, 513, "tree", True, 0)])
def test_verify_tree_matches(B, T, V, shape, draft, pad):
    g = torch.Generator().manual_seed(B + T + V)
    for k in range(4):
        p, q, tok, par, n, ua, us = verify_inputs(B, T, V, g, shape, pad, noise=0.4 * (k + 1))
        ref = TO.verify_tree(p[..., :V].numpy(), q[..., :V].numpy() if draft else None, tok.numpy(), par.numpy(), n.numpy(), ua.numpy(),
                             us.numpy())
        got = run_verify(p, q if draft else None, tok, par, n, ua, us, V)
        for x, y in zip(got, ref):
            assert np.array_equal(x, y), (k, x, y)


def test_verify_tree_borders_and_masses():
    """Dyadic rows whose sums are exact: a draw on a border takes the next entry with mass, u = 0 the first; a target equal to the
    draft always stands; a one-hot target stands on its token alone; nothing left falls back on the row; no mass at all: -1."""
    V = 8
    p = torch.zeros(6, 2, V)
    p[0, 1] = torch.tensor([0, .25, 0, .25, .25, 0, .25, 0])
    p[1, 1] = p[0, 1]
    p[2, 0] = torch.tensor([0, 0, .5, .5, 0, 0, 0, 0])
    p[2, 1, 7] = 1.0
    p[3, 0, 4] = 1.0
    p[3, 1, 5] = 1.0
    p[4, 0, 6] = 1.0
    p[5, 0] = float("nan")
    q = torch.full((6, 2, V), 1 / 8)
    p[0, 0] = p[1, 0] = 1 / 8
    q[4, 0] = p[4, 0]
    tok = torch.tensor([[0, 3], [0, 5], [0, 3], [0, 2], [0, 1], [0, 2]], dtype=I32)
    par = torch.tensor([[-1, 0]] * 6, dtype=I32)
    n = torch.full((6,), 2, dtype=I32)
    ua = torch.tensor([[.0, .999], [.0, .999], [.0, .999], [.0, .0], [.0, .0], [.0, .0]])
    us = torch.tensor([.5, 0., .999, .5, .5, .5])
    path, cnt, nxt = run_verify(p, q, tok, par, n, ua, us, V)
    ref = TO.verify_tree(p.numpy(), q.numpy(), tok.numpy(), par.numpy(), n.numpy(), ua.numpy(), us.numpy())
    assert cnt.tolist() == [2, 2, 2, 1, 1, 1] and nxt.tolist() == [4, 1, 7, 4, 6, -1]
    for x, y in zip((path, cnt, nxt), ref):
        assert np.array_equal(x, y)


def test_verify_tree_same_token_twice_and_bad_tokens():
    V, T = 16, 6
    g = torch.Generator().manual_seed(9)
    p = torch.softmax(torch.randn(1, T, V, generator=g), -1)
    par = torch.tensor([[-1, 0, 0, 0, 0, 0]], dtype=I32)
    tok = torch.tensor([[0, 3, 3, 3, 3, 3]], dtype=I32)
    n = torch.tensor([T], dtype=I32)
    ua, us = torch.full((1, T), 0.999), torch.tensor([0.3])
    ref = TO.verify_tree(p.numpy(), None, tok.numpy(), par.numpy(), n.numpy(), ua.numpy(), us.numpy())
    for x, y in zip(run_verify(p, None, tok, par, n, ua, us, V), ref):
        assert np.array_equal(x, y)
    assert ref[1][0] == 1 and ref[2][0] != 3
    assert lsk.read_device_error(clear=True) == 0
    tok[0, 1], tok[0, 2], par[0, 3], par[0, 4] = 16, -1, 4, -7
    got = run_verify(p, None, tok, par, n, torch.zeros(1, T), us, V)
    assert got[1][0] == 2 and got[0][0].tolist() == [0, 5, -1, -1, -1, -1]
    assert lsk.read_device_error(clear=True) == lsk.DEVERR_ID_RANGE


@pytest.mark.parametrize("draft", [True, False])
def test_verify_tree_entries_that_are_no_probabilities(draft):
    """Negative, infinite, NaN and subnormal entries in both rows, at nodes that reject, accept and draw: all but the subnormal ones
    count as 0."""
    B, T, V = 6, 9, 1201
    g = torch.Generator().manual_seed(21)
    p, q, tok, par, n, ua, us = verify_inputs(B, T, V, g, "tree", 0, noise=1.5, ragged=False)
    for k, x in enumerate((float("inf"), float("-inf"), float("nan"), -0.25, -0.0, 1e-42)):
        for t in (p, q):
            at = torch.randint(0, V, (B, T, 5), generator=g)
            t[..., :V].scatter_(2, at, x)
    ref = TO.verify_tree(p.numpy(), q.numpy() if draft else None, tok.numpy(), par.numpy(), n.numpy(), ua.numpy(), us.numpy())
    got = run_verify(p, q if draft else None, tok, par, n, ua, us, V)
    for x, y in zip(got, ref):
        assert np.array_equal(x, y), (x, y)


def test_verify_tree_draws_with_the_targets_frequencies():
    """A chain of one draft over 4 tokens, 40,000 sequences: next tokens (the draft where it stands, else the draw) follow the
    target.  Counts are binomial: 5 standard deviations of 40,000 p (1 - p)."""
    B, V = 40000, 4
    g = torch.Generator().manual_seed(4)
    pt, pd = torch.tensor([.5, .25, .2, .05]), torch.tensor([.1, .2, .3, .4])
    p, q = pt.repeat(B, 2, 1), pd.repeat(B, 2, 1)
    tok = torch.multinomial(pd, B, True, generator=g).int()
    tokens = torch.stack([torch.zeros(B, dtype=I32), tok], 1)
    par = torch.tensor([[-1, 0]], dtype=I32).repeat(B, 1)
    ua, us = torch.rand(B, 2, generator=g), torch.rand(B, generator=g)
    path, cnt, nxt = run_verify(p, q, tokens, par, torch.full((B,), 2, dtype=I32), ua, us, V)
    first = np.where(cnt == 2, tok.numpy(), nxt)
    for x in range(V):
        e = float(pt[x])
        assert abs((first == x).sum() - B * e) <= 5 * math.sqrt(B * e * (1 - e))


# ------------------------------------------------------------------------------------------ commit_path

def commit_case(L, B, H, K, N, T, seed, ctx=None, n=None):
    g = torch.Generator().manual_seed(seed)
    host = torch.randn(L, B, H, N, 2, 16, 128, generator=g).to(BF).pin_memory()
    st = torch.stack([torch.randperm(N, generator=g)[:K] for _ in range(L * B * H)]).view(L, B, H, K).int()
    st[torch.rand(L, B, H, K, generator=g) < 0.2] = -1
    pool = torch.randn(L, B, H, K, 2, 16, 128, generator=g).to(BF)
    kmin, kmax = host[..., 0, :, :].float().amin(-2).to(BF), host[..., 0, :, :].float().amax(-2).to(BF)
    k, v = (torch.randn(L, B, H, T, 128, generator=g).to(BF) * 2 for _ in range(2))
    count = torch.tensor(n if n is not None else [int(torch.randint(0, T + 1, (1,), generator=g)) for _ in range(B)], dtype=I32)
    path = torch.full((B, T), -1, dtype=I32)
    for b in range(B):
        path[b, :count[b]] = torch.randperm(T, generator=g)[:count[b]].sort().values.int()
    c = torch.tensor(ctx if ctx is not None else [int(torch.randint(0, N * 16 - T + 1, (1,), generator=g)) for _ in range(B)], dtype=I32)
    return host, pool, st, kmin, kmax, k, v, path, count, c


@pytest.mark.parametrize("L,B,H,K,N,T,ctx,n", [
    (1, 1, 1, 1, 4, 1, [0], [1]), (1, 2, 2, 4, 8, 5, [14, 16], [5, 5]), (3, 3, 2, 6, 12, 8, None, None),
    (2, 2, 1, 12, 12, 64, [5, 128], [64, 64]), (70, 2, 1, 3, 6, 4, None, None), (1, 4, 2, 4, 8, 16, [15, 0, 112, 17], [0, 16, 16, 1])])
@pytest.mark.parametrize("parts", ["all", "no_host", "no_pool"])
def test_commit_path_matches(L, B, H, K, N, T, ctx, n, parts):
    host, pool, st, kmin, kmax, k, v, path, count, c = commit_case(L, B, H, K, N, T, L + T, ctx, n)
    ref = {x: f64(t) for x, t in (("host", host), ("pool", pool), ("kmin", kmin), ("kmax", kmax))}
    want = TO.commit_path(ref["host"] if parts != "no_host" else None, ref["pool"] if parts != "no_pool" else None, st.numpy(),
                          ref["kmin"], ref["kmax"], f64(k), f64(v), path.numpy(), count.numpy(), c.numpy())
    d = lsk.make_dims(B, H, H, N, K, 1, 0)
    pool, st, kmin, kmax, k, v = (t.to(DEV) for t in (pool, st, kmin, kmax, k, v))
    layers = lsk.make_cache_layers(d, None if parts == "no_host" else host, kmin, kmax, st, None if parts == "no_pool" else pool)
    out = torch.full((B,), -1, dtype=I32, device=DEV)
    for _ in range(2):                             # a second call at the same lengths writes the same
        lsk.commit_path(d, T, layers, k, v, path.to(DEV), count.to(DEV), c.to(DEV), out)
        torch.cuda.synchronize()
        for name, t in (("host", host), ("pool", pool), ("kmin", kmin), ("kmax", kmax)):
            assert np.array_equal(f64(t), ref[name]), name
        assert out.tolist() == want.tolist()


def test_commit_path_equals_appends():
    """A chain committed at once leaves what appending its tokens one by one leaves."""
    host, pool, st, kmin, kmax, k, v, path, count, c = commit_case(1, 2, 2, 6, 8, 7, 5, [30, 12], [7, 7])
    d = lsk.make_dims(2, 2, 2, 8, 6, 1, 0)
    bufs = [t.to(DEV) for t in (pool[0], kmin[0], kmax[0])]
    host2 = host.clone().pin_memory()
    ctx = [c.to(DEV), c.to(DEV).clone()]
    std = st[0].contiguous().to(DEV)
    for t in range(7):
        lsk.append_kv(d, k[0, :, :, t].contiguous().to(DEV), v[0, :, :, t].contiguous().to(DEV), ctx[t % 2], ctx[1 - t % 2], host2[0], bufs[1],
                      bufs[2], std, bufs[0])
    pool, kmin, kmax = (t.to(DEV) for t in (pool, kmin, kmax))
    out = torch.empty(2, dtype=I32, device=DEV)
    layer = lsk.make_layer(d, host[0], kmin[0], kmax[0], pool[0], std, torch.zeros_like(std), torch.zeros_like(std), None, None,
                           None, None, torch.zeros(4, dtype=I32, device=DEV), torch.zeros(2, 1, 2, 128, device=DEV),
                           torch.zeros(2, 1, 2, device=DEV))
    lsk.commit_path(d, 7, [layer], k.to(DEV), v.to(DEV), path.to(DEV), count.to(DEV), c.to(DEV), out)
    torch.cuda.synchronize()
    assert torch.equal(host, host2) and torch.equal(pool[0], bufs[0]) and torch.equal(kmin[0], bufs[1]) and torch.equal(kmax[0], bufs[2])
    assert torch.equal(out, ctx[1])


def test_commit_path_flags_full_caches_and_bad_ids():
    host, pool, st, kmin, kmax, k, v, path, count, c = commit_case(1, 3, 1, 4, 4, 6, 8, [61, 64, 10], [6, 2, 3])
    path[2, 1] = 6
    keep = host.clone()
    d = lsk.make_dims(3, 1, 1, 4, 4, 1, 0)
    pool, st, kmin, kmax, k, v = (t.to(DEV) for t in (pool, st, kmin, kmax, k, v))
    layers = lsk.make_cache_layers(d, host, kmin, kmax, st, pool)
    out = torch.empty(3, dtype=I32, device=DEV)
    lsk.commit_path(d, 6, layers, k, v, path.to(DEV), count.to(DEV), c.to(DEV), out)
    assert lsk.read_device_error(clear=True) == lsk.DEVERR_APPEND_FULL | lsk.DEVERR_ID_RANGE
    assert out.tolist() == [64, 64, 13]
    kc = k.cpu()
    keep[0, 0, 0, 3, 0, 13:], keep[0, 0, 0, 3, 1, 13:] = kc[0, 0, 0, path[0, :3].long()], v.cpu()[0, 0, 0, path[0, :3].long()]
    for i in (0, 2):
        keep[0, 2, 0, 0, 0, 10 + i], keep[0, 2, 0, 0, 1, 10 + i] = kc[0, 2, 0, path[2, i]], v.cpu()[0, 2, 0, path[2, i]]
    assert torch.equal(host, keep)
    count[0] = 99
    lsk.commit_path(d, 6, layers, k, v, path.clamp(0, 5).to(DEV), count.to(DEV), torch.zeros(3, dtype=I32, device=DEV), out)
    assert lsk.read_device_error(clear=True) == lsk.DEVERR_ID_RANGE and out.tolist() == [6, 2, 3]
