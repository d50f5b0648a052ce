"""The draft-tree calls as a program runs them: speculative steps over a small two-layer decoder and the sparse KV pipeline, each
result held against the fp64 statements on the tensors the step itself used; the same calls captured into a graph; two streams."""

import numpy as np
import pytest
import torch

import lookahead_sparse_kv_b200 as lsk
from lookahead_sparse_kv_b200 import workloads as W
from lookahead_sparse_kv_b200.pipeline import DecodePipeline, LayerState, TreeDecoder
from oracle import bf16_bits_to_f64
from oracle import tree_oracle as TO

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, I32 = torch.bfloat16, torch.int32
L, B, HQ, HKV, K, N, V, WIDE = 2, 3, 8, 2, 24, 40, 307, 96


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from lookahead_sparse_kv_b200 import build
    build.build()
    lsk.lib()
    yield
    assert lsk.read_device_error(clear=True) == 0


def f64(t):
    return bf16_bits_to_f64(W.bf16_bits(t))


def close(got, ref, size):
    """bf16 weights and a bf16 store, as in the attention's own tests: 2^-8 |o| + (2^-8 + 2^-16) A."""
    return not bool((np.abs(got - ref) > 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -16) * size + 1e-30).any())


def small_model(g):
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"emb": r(V, WIDE).to(BF).to(DEV), "qkv": [(r(WIDE, (HQ + 2 * HKV) * 128) * 0.2).to(BF).to(DEV) for _ in range(L)],
            "o": [(r(HQ * 128, WIDE) * 0.05).to(BF).to(DEV) for _ in range(L)], "head": (r(WIDE, V) * 0.3).to(BF).to(DEV),
            "w": [[(1 + 0.1 * r(128)).to(BF).to(DEV) for _ in range(L)] for _ in range(2)]}


@pytest.mark.parametrize("T", [8, 21])
def test_speculative_steps(T):
    g = torch.Generator().manual_seed(T)
    M = small_model(g)
    Qn = 8
    d = lsk.make_dims(B, HQ, HKV, N, K, Qn, 6)
    hosts = [torch.randn(B, HKV, N, 2, 16, 128, generator=g).to(BF).pin_memory() for _ in range(L)]
    layers = [LayerState(d, h) for h in hosts]
    ctx0 = torch.tensor([77, 301, 16], dtype=I32)
    pipe = DecodePipeline(d, layers, ctx0.to(DEV), 128 ** -0.5)
    pipe.build_summaries()
    pipe.prime([torch.randn(B, Qn, HQ, 128, generator=g).to(BF).to(DEV) for _ in range(L)])
    inv = (1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(DEV)
    dec = TreeDecoder(pipe, T, inv, wq=M["w"][0], wk=M["w"][1])
    ctx = ctx0.numpy().copy()
    for step in range(3):
        j = torch.arange(T).repeat(B, 1)
        parent = torch.where(j > 0, (torch.rand(B, T, generator=g) * j).floor().long(), -1).int()
        n = torch.tensor([T, T - 3, T], dtype=I32)
        tokens = torch.randint(0, V, (B, T), generator=g).int()
        ua, us = torch.rand(B, T, generator=g), torch.rand(B, generator=g)
        dec.begin(parent.to(DEV), n.to(DEV))
        x = M["emb"][tokens.to(DEV).long()]
        mask, pos = TO.tree_layout(parent.numpy(), n.numpy(), ctx)
        for i, S in enumerate(layers):
            qkv = x @ M["qkv"][i]
            torch.cuda.synchronize()
            st, pool = S.slot_table.cpu().numpy(), f64(S.pool)          # what the attention will see
            out = dec.layer(i, qkv)
            torch.cuda.synchronize()
            assert np.array_equal(dec.mask.cpu().numpy().view(np.uint64), mask) and np.array_equal(dec.pos.cpu().numpy(), pos)
            q, k, v = TO.qk_norm_rope(f64(qkv).reshape(B, T, HQ + 2 * HKV, 128), HQ, HKV, f64(M["w"][0][i]), f64(M["w"][1][i]), 1e-6,
                                      inv.cpu().numpy(), pos)
            for got, ref in ((dec.q, q), (dec.k_tree[i], k), (dec.v_tree[i], v)):
                length = np.hypot(ref[..., :64], ref[..., 64:])
                assert bool((np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * np.concatenate([length, length], -1)).all())
            a = (f64(dec.q), pool[:, :, :, 0], pool[:, :, :, 1], st, ctx, f64(dec.k_tree[i]), f64(dec.v_tree[i]), mask, pipe.scale)
            ref, _ = TO.tree_attention(*a)
            size, _ = TO.tree_attention(a[0], a[1], np.abs(a[2]), a[3], a[4], a[5], np.abs(a[6]), *a[7:])
            assert close(f64(out), ref, size)
            x = x + out.flatten(2) @ M["o"][i]
        probs = torch.softmax(x.float() @ M["head"].float(), -1)
        # the drafts came from a flattened copy of the target
        draft = torch.softmax(0.7 * torch.log(probs), -1)
        nxt = dec.verify(probs, tokens.to(DEV), ua.to(DEV), us.to(DEV), draft)
        path, cnt, tok = TO.verify_tree(probs.cpu().numpy(), draft.cpu().numpy(), tokens.numpy(), parent.numpy(), n.numpy(), ua.numpy(),
                                        us.numpy())
        assert np.array_equal(dec.path.cpu().numpy(), path) and np.array_equal(dec.n_accept.cpu().numpy(), cnt)
        assert np.array_equal(nxt.cpu().numpy(), tok) and cnt.min() >= 1
        torch.cuda.synchronize()
        before = [{"host": f64(S.host_kv)[None], "pool": f64(S.pool)[None], "kmin": f64(S.kmin)[None], "kmax": f64(S.kmax)[None],
                   "st": S.slot_table.cpu().numpy()[None]} for S in layers]
        dec.commit()
        torch.cuda.synchronize()
        for i, (S, b) in enumerate(zip(layers, before)):
            after = TO.commit_path(b["host"], b["pool"], b["st"], b["kmin"], b["kmax"], f64(dec.k_tree[i:i + 1]), f64(dec.v_tree[i:i + 1]),
                                   path, cnt, ctx)
            assert np.array_equal(f64(S.host_kv), b["host"][0]) and np.array_equal(f64(S.pool), b["pool"][0])
            assert np.array_equal(f64(S.kmin), b["kmin"][0]) and np.array_equal(f64(S.kmax), b["kmax"][0])
        ctx = after
        assert pipe.ctx_len.tolist() == ctx.tolist()


def one_step(d, T, s, stream=None):
    """The five calls over the tensors of `s`, in stream order."""
    lsk.tree_layout(d, T, s["parent"], s["n"], s["ctx"], s["mask"], s["pos"], stream=stream)
    lsk.qk_norm_rope(d, T, s["qkv"], s["w"], s["w"], 1e-6, s["inv"], s["pos"], s["q"], s["k"][0], s["v"][0], stream=stream)
    lsk.tree_attn(d, T, s["q"], s["pool"][0], s["st"][0], s["ctx"], s["k"][0], s["v"][0], s["mask"], 0.09, s["out"], s["lse"], s["ws"], stream=stream)
    lsk.verify_tree(d, T, s["probs"], s["draft"], s["tokens"], s["parent"], s["n"], s["ua"], s["us"], s["path"], s["cnt"], s["next"], stream=stream)
    lsk.commit_path(d, T, s["layers"], s["k"], s["v"], s["path"], s["cnt"], s["ctx"], s["ctx_out"], stream=stream)


def step_tensors(d, T, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)  # noqa: E731
    j = torch.arange(T).repeat(B, 1)
    s = {"parent": torch.where(j > 0, (torch.rand(B, T, generator=g) * j).floor().long(), -1).int().to(DEV),
         "n": torch.tensor([T, 0, T // 2 + 1], dtype=I32, device=DEV), "ctx": torch.tensor([300, 40, 5], dtype=I32, device=DEV),
         "mask": torch.empty(B, T, dtype=torch.uint64, device=DEV), "pos": torch.empty(B, T, dtype=I32, device=DEV),
         "qkv": r(B, T, (HQ + 2 * HKV) * 128), "w": r(128), "inv": torch.rand(64, generator=g).to(DEV), "q": r(B, T, HQ, 128),
         "k": r(1, B, HKV, T, 128), "v": r(1, B, HKV, T, 128), "pool": r(1, B, HKV, K, 2, 16, 128), "out": r(B, T, HQ, 128),
         "st": torch.stack([torch.randperm(N, generator=g)[:K] for _ in range(B * HKV)]).view(1, B, HKV, K).int().to(DEV),
         "lse": torch.zeros(B, T, HQ, device=DEV), "kmin": r(1, B, HKV, N, 128), "kmax": r(1, B, HKV, N, 128),
         "host": torch.randn(1, B, HKV, N, 2, 16, 128, generator=g).to(BF).pin_memory(),
         "probs": torch.softmax(3 * torch.randn(B, T, V, generator=g), -1).to(DEV), "draft": torch.softmax(3 * torch.randn(B, T, V, generator=g), -1).to(DEV),
         "tokens": torch.randint(0, V, (B, T), generator=g).int().to(DEV), "ua": torch.rand(B, T, generator=g).to(DEV) * 0.3,
         "us": torch.rand(B, generator=g).to(DEV), "path": torch.empty(B, T, dtype=I32, device=DEV), "cnt": torch.empty(B, dtype=I32, device=DEV),
         "next": torch.empty(B, dtype=I32, device=DEV), "ctx_out": torch.empty(B, dtype=I32, device=DEV),
         "ws": torch.full((lsk.tree_workspace_bytes(d, T),), 255, dtype=torch.uint8, device=DEV)}
    s["layers"] = lsk.make_cache_layers(d, s["host"], s["kmin"], s["kmax"], s["st"], s["pool"])
    return s


RESULTS = ("mask", "pos", "q", "k", "v", "out", "lse", "path", "cnt", "next", "ctx_out", "kmin", "kmax", "pool", "host")


def results(s):
    torch.cuda.synchronize()
    return {n: s[n].cpu().clone() for n in RESULTS}


def same(a, b):
    return all(torch.equal(a[n].view(torch.int64) if a[n].dtype == torch.uint64 else a[n],
                           b[n].view(torch.int64) if b[n].dtype == torch.uint64 else b[n]) for n in RESULTS)


@pytest.mark.parametrize("T", [5, 64])
def test_captured_and_replayed(T):
    """One step captured as a graph, replayed on other inputs written into its buffers: the eager calls' bits.  The workspace starts
    as garbage and is shared by both."""
    d = lsk.make_dims(B, HQ, HKV, N, K, 1, 0)
    first, other = step_tensors(d, T, 1), step_tensors(d, T, 2)
    one_step(d, T, other)
    want = results(other)
    stream = torch.cuda.Stream()
    one_step(d, T, first)                              # (warm: launch attributes are set once)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        one_step(d, T, first)
    again = step_tensors(d, T, 2)
    for n in first:
        if isinstance(first[n], torch.Tensor) and n != "ws":
            first[n].copy_(again[n])
    torch.cuda.synchronize()
    for _ in range(3):                                 # the same lengths: every replay writes the same
        graph.replay()
    assert same(results(first), want)


def test_two_streams_at_once():
    """Two independent steps on two streams, interleaved call by call, give what each gives alone."""
    T = 17
    d = lsk.make_dims(B, HQ, HKV, N, K, 1, 0)
    want = []
    for seed in (3, 4):
        s = step_tensors(d, T, seed)
        one_step(d, T, s)
        want.append(results(s))
    both = [step_tensors(d, T, seed) for seed in (3, 4)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, stream in zip(both, streams):
            with torch.cuda.stream(stream):
                one_step(d, T, s)                      # (the current stream)
    torch.cuda.synchronize()
    for s, w in zip(both, want):
        assert same(results(s), w)
    for s, stream in zip(both, streams):
        one_step(d, T, s, stream=stream)               # (a stream given by name)
    torch.cuda.synchronize()
    for s, w in zip(both, want):
        assert same(results(s), w)
