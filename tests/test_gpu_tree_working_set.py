"""The working set under a TreeDecoder: selection, plan, LRU order and gather of tree steps mixed with plain decode steps, against the
oracle; and whole steps with no host synchronisation inside, on two streams against one."""

import numpy as np
import pytest
import torch

import lookahead_sparse_kv_b200 as lsk
import oracle as O
from lookahead_sparse_kv_b200 import workloads as W
from lookahead_sparse_kv_b200.pipeline import DecodePipeline, LayerState, TreeDecoder
from tests.gpu_util import assert_selection_matches, f64, np_i32

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, I32 = torch.bfloat16, torch.int32
V = 211


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from lookahead_sparse_kv_b200 import build
    build.build()
    lsk.lib()
    yield
    assert lsk.read_device_error(clear=True) == 0


def tree_inputs(B, T, width, layers, g):
    """Parents, projection rows per layer and the verification's inputs of one step."""
    j = torch.arange(T).repeat(B, 1)
    return {"parent": torch.where(j > 0, (torch.rand(B, T, generator=g) * j).floor().long(), -1).int().to(DEV),
            "qkv": [torch.randn(B, T, width, generator=g).to(BF).to(DEV) for _ in range(layers)],
            "probs": torch.softmax(2 * torch.randn(B, T, V, generator=g), -1).to(DEV),
            "tokens": torch.randint(0, V, (B, T), generator=g).int().to(DEV), "ua": (0.2 * torch.rand(B, T, generator=g)).to(DEV),
            "us": torch.rand(B, generator=g).to(DEV)}


def tree_step(dec, s, keep):
    """One step; keep(i, out) after each layer's call.  Nothing waits on the host."""
    dec.begin(s["parent"])
    for i, qkv in enumerate(s["qkv"]):
        keep(i, dec.layer(i, qkv))
    dec.verify(s["probs"], s["tokens"], s["ua"], s["us"])
    dec.commit()


@pytest.mark.parametrize("again", [False, True])
def test_lru_order_over_tree_and_plain_steps(again):
    """Plain steps, tree steps of one width, then another, plain steps again (and, with `again`, a second priming): every plan is the
    oracle's for a step number that only grows, so the least recently used blocks go, whichever kind of step used them."""
    L, B, HQ, HKV, K, N, Qn, cap = 2, 2, 8, 2, 12, 64, 4, 5
    g = torch.Generator().manual_seed(17)
    d = lsk.make_dims(B, HQ, HKV, N, K, Qn, cap)
    layers = [LayerState(d, torch.randn(B, HKV, N, 2, 16, 128, generator=g).to(BF).pin_memory()) for _ in range(L)]
    ctx = torch.tensor([900, 640], dtype=I32)
    pipe = DecodePipeline(d, layers, ctx.to(DEV), 128 ** -0.5)
    pipe.build_summaries()
    inv = torch.full((64,), 0.01, device=DEV)
    decs = {T: TreeDecoder(pipe, T, inv) for T in (4, 9)}
    state = [(np_i32(S.slot_table), np_i32(S.last_used)) for S in layers]
    stamp = 0

    def check(rows, ctx_now, maps):
        """Each layer's selection from the query rows and summaries that the plan saw, and its plan from the oracle's own state."""
        torch.cuda.synchronize()
        for i, S in enumerate(layers):
            sel = np_i32(S.sel)
            sc = O.lookahead_scores(f64(rows[i]), *maps[i], ctx_now, 16)
            assert_selection_matches(sel, O.select_topk(sc, ctx_now, K, 16)[0], sc, ctx_now, K)
            plan = O.plan_fetch(sel, *state[i], stamp, cap)
            state[i] = (plan["slot_table"], plan["last_used"])
            for name in ("n_fetch", "fetch_block", "slot_table", "last_used"):
                np.testing.assert_array_equal(np_i32(getattr(S, name)), plan[name], err_msg=f"{name}, layer {i}, step {stamp}")
            host, pool = W.bf16_bits(S.host_kv), W.bf16_bits(S.pool)
            for b, h, s in zip(*np.nonzero(plan["slot_table"] >= 0)):
                np.testing.assert_array_equal(pool[b, h, s], host[b, h, plan["slot_table"][b, h, s]])

    def summaries():
        torch.cuda.synchronize()
        return [(f64(S.kmin), f64(S.kmax)) for S in layers]

    def queries():
        return [torch.randn(B, Qn, HQ, 128, generator=g).to(BF).to(DEV) for _ in range(L)]

    t = 0
    steps = ["prime", *["plain"] * 5, *[4] * 2, *[9] * 2, *["plain"] * 3, 4, 9, "plain"]
    for kind in steps + (steps[:8] if again else []):
        maps, now = summaries(), pipe.ctx_len.cpu().numpy().copy()
        if kind == "prime":
            rows = queries()
            pipe.prime(rows)
            t = 0
        elif kind == "plain":
            rows, t = queries(), t + 1
            pipe.step(t, rows)
        else:
            rows = [None] * L
            dec = decs[kind]

            def keep(i, out):
                rows[i] = dec.q[:, :Qn].clone()
            tree_step(dec, tree_inputs(B, kind, (HQ + 2 * HKV) * 128, L, g), keep)
        check(rows, now, maps)
        stamp += 1


def run_steps(single, steps, T):
    """Tree steps, a plain step between them, on a pool whose gathers outlast the attention; the results, cloned in stream order."""
    L, B, HQ, HKV, K, N, Qn, cap = 2, 2, 16, 4, 128, 512, 4, 96
    g = torch.Generator().manual_seed(T)
    d = lsk.make_dims(B, HQ, HKV, N, K, Qn, cap)
    layers = [LayerState(d, torch.randn(B, HKV, N, 2, 16, 128, generator=g).to(BF).pin_memory()) for _ in range(L)]
    pipe = DecodePipeline(d, layers, torch.tensor([8100, 5000], dtype=I32, device=DEV), 128 ** -0.5, single_stream=single)
    pipe.build_summaries()
    pipe.prime([torch.randn(B, Qn, HQ, 128, generator=g).to(BF).to(DEV) for _ in range(L)])
    dec = TreeDecoder(pipe, T, torch.full((64,), 0.01, device=DEV))
    inputs = [tree_inputs(B, T, (HQ + 2 * HKV) * 128, L, g) for _ in range(steps)]
    plain = [torch.randn(B, Qn, HQ, 128, generator=g).to(BF).to(DEV) for _ in range(L)]
    torch.cuda.synchronize()
    got = []
    for n, s in enumerate(inputs):
        tree_step(dec, s, lambda i, out: got.extend((out.clone(), dec.lse.clone())))
        got.extend((dec.path.clone(), dec.n_accept.clone(), dec.next_token.clone(), pipe.ctx_len.clone()))
        if n == 1:
            pipe.step(1, plain)
            got.extend(S.out.clone() for S in layers)
    pipe.wait_all()
    torch.cuda.synchronize()
    for S in layers:
        got.extend((S.pool, S.slot_table, S.last_used, S.kmin, S.kmax, S.host_kv))
    return [t.cpu() for t in got]


@pytest.mark.parametrize("T", [4, 13])
def test_steps_without_host_waits_match_one_stream(T):
    """Attention waits for the gather that the last step planned and a commit for the gathers of its own, whatever the host does."""
    two, one = run_steps(False, 4, T), run_steps(True, 4, T)
    for i, (a, b) in enumerate(zip(two, one)):
        assert torch.equal(a, b), i
