"""The draft-tree calls turn bad arguments down on the host: the library's own checks (raw addresses that are never read) and the
binding's (dtype, layout, size, device).  CPU only."""

import ctypes

import pytest
import torch

import lookahead_sparse_kv_b200 as lsk
from lookahead_sparse_kv_b200 import build as lsk_build

A = 16                                # an aligned address that no check reads
NAMES = ["tree_layout", "qk_norm_rope", "tree_attn", "verify_tree", "commit_path"]


@pytest.fixture(scope="module")
def L():
    lsk_build.build()
    return lsk.lib()


def dims(**kw):
    return lsk.make_dims(**{**dict(batch=2, n_q_heads=8, n_kv_heads=2, max_blocks=64, budget_blocks=16, n_queries=5, fetch_cap=4), **kw})


def layer(**kw):
    at = dict(host_kv=0, kmin=A, kmax=A, pool=0, slot_table=0)
    return (lsk.Layer * 1)(lsk.Layer(**{**at, **kw}))


def call(L, name, d=None, **kw):
    """The named entry point with sound raw arguments, some of them replaced."""
    big = 1 << 40
    args = {
        "tree_layout": dict(n_tree=5, parent=A, n_nodes=A, ctx_len=A, mask=A, pos=A),
        "qk_norm_rope": dict(n_tok=5, qkv=A, row_stride=12 * 128, wq=A, wk=A, eps=1e-6, inv_freq=A, pos=A, q=A, k=A, v=A),
        "tree_attn": dict(n_tree=5, q=A, pool=A, slot_table=A, ctx_len=A, k_tree=A, v_tree=A, mask=A, scale=0.1, out=A, lse=A, ws=A,
                          ws_bytes=big),
        "verify_tree": dict(n_tree=5, vocab=100, probs=A, draft=A, row_stride=100, tokens=A, parent=A, n_nodes=A, u_accept=A, u_sample=A,
                            path=A, n_accept=A, next_token=A),
        "commit_path": dict(n_tree=5, layers=layer(), n_layers=1, k_tree=A, v_tree=A, path=A, n_accept=A, ctx_len=A, ctx_len_out=2 * A),
    }[name]
    assert set(kw) <= set(args)
    args.update(kw)
    d = dims() if d is None else d
    rc = getattr(L, "oasis_" + name)(ctypes.byref(d), *args.values(), None)
    return rc, lsk.last_error()


@pytest.mark.parametrize("name,arg,value,says", [
    ("tree_layout", "n_tree", 0, "n_tree"), ("tree_layout", "n_tree", 65, "n_tree"), ("tree_layout", "parent", None, "parent is NULL"),
    ("tree_layout", "mask", 8, "mask is not 16-byte"), ("tree_layout", "pos", None, "pos"), ("tree_layout", "ctx_len", None, "ctx_len"),
    ("qk_norm_rope", "n_tok", 0, "n_tok"), ("qk_norm_rope", "row_stride", 12 * 128 - 8, "row_stride"),
    ("qk_norm_rope", "row_stride", 12 * 128 + 4, "row_stride"), ("qk_norm_rope", "eps", -1.0, "eps"),
    ("qk_norm_rope", "eps", float("nan"), "eps"), ("qk_norm_rope", "inv_freq", None, "inv_freq"), ("qk_norm_rope", "q", 24, "q is not"),
    ("qk_norm_rope", "wq", 24, "wq is not"),
    ("tree_attn", "n_tree", -1, "n_tree"), ("tree_attn", "n_tree", 65, "n_tree"), ("tree_attn", "scale", 0.0, "scale"),
    ("tree_attn", "scale", float("inf"), "scale"), ("tree_attn", "scale", float("nan"), "scale"), ("tree_attn", "mask", None, "mask"),
    ("tree_attn", "v_tree", None, "v_tree"), ("tree_attn", "ws", None, "ws"), ("tree_attn", "ws_bytes", 100, "workspace"),
    ("verify_tree", "vocab", 0, "vocab"), ("verify_tree", "vocab", (1 << 30) + 1, "vocab"), ("verify_tree", "row_stride", 99, "row_stride"),
    ("verify_tree", "probs", None, "probs"), ("verify_tree", "probs", 20, "probs is not"), ("verify_tree", "draft", 20, "draft_probs"),
    ("verify_tree", "u_sample", None, "u_sample"), ("verify_tree", "next_token", None, "next_token"), ("verify_tree", "n_tree", 0, "n_tree"),
    ("commit_path", "n_layers", 0, "n_layers"), ("commit_path", "layers", None, "layers"), ("commit_path", "path", None, "path"),
    ("commit_path", "ctx_len_out", A, "alias"), ("commit_path", "n_tree", 99, "n_tree"),
])
def test_library_turns_down(L, name, arg, value, says):
    rc, msg = call(L, name, **{arg: value})
    assert rc == lsk.EINVAL and says in msg, (rc, msg)


@pytest.mark.parametrize("kw,says", [(dict(kmin=0), "kmin"), (dict(kmax=24), "kmax"), (dict(pool=A, slot_table=0), "slot_table is NULL"),
                                     (dict(pool=A, slot_table=2), "4-byte"), (dict(pool=24), "pool"), (dict(host_kv=24), "host_kv")])
def test_library_turns_down_bad_layers(L, kw, says):
    rc, msg = call(L, "commit_path", layers=layer(**kw))
    assert rc == lsk.EINVAL and says in msg, (rc, msg)


@pytest.mark.parametrize("name", NAMES)
def test_library_turns_down_bad_dims(L, name):
    rc, msg = call(L, name, d=dims(head_dim=64))
    assert rc == lsk.EINVAL and "head_dim" in msg
    assert lsk.tree_workspace_bytes(dims(head_dim=64), 5) == 0 and lsk.tree_workspace_bytes(dims(), 0) == 0
    assert lsk.tree_workspace_bytes(dims(), 65) == 0


def test_too_many_heads_a_kv_head(L):
    d = dims(n_q_heads=66, n_kv_heads=1, n_queries=1)
    assert lsk.check_dims(d) == lsk.EINVAL                        # 66 query rows even for one position
    assert lsk.tree_workspace_bytes(d, 1) == 0


def test_workspace_does_not_grow_with_the_batch(L):
    """Two places a CTA, whatever the batch."""
    one = lsk.tree_workspace_bytes(dims(), 64)
    assert one == lsk.tree_workspace_bytes(dims(batch=64), 64) > 0


def err(fn):
    with pytest.raises(lsk.OasisError) as e:
        fn()
    assert e.value.code == lsk.EINVAL
    return str(e.value)


def test_binding_turns_down_tensors_that_do_not_fit():
    d = dims()
    B, T, V = 2, 5, 100
    i = torch.zeros(B, T, dtype=torch.int32)
    m = torch.zeros(B, T, dtype=torch.int64)
    assert "parent must be int32" in err(lambda: lsk.tree_layout(d, T, i.long(), None, A, A, A))
    assert "parent must be on a CUDA device" in err(lambda: lsk.tree_layout(d, T, i, None, A, A, A))
    assert "parent holds" in err(lambda: lsk.tree_layout(d, T + 1, i, None, A, A, A))
    assert "parent must be contiguous" in err(lambda: lsk.tree_layout(d, T, i.t(), None, A, A, A))
    assert "parent is None" in err(lambda: lsk.tree_layout(d, T, None, None, A, A, A))
    assert "n_tree" in err(lambda: lsk.tree_layout(d, 65, i, None, A, A, A))
    assert "mask must be int64" in err(lambda: lsk.tree_layout(d, T, A, None, A, m.int(), A))
    assert "mask must be on a CUDA device" in err(lambda: lsk.tree_layout(d, T, A, None, A, m, A))
    rows = torch.zeros(B, T, 12 * 128, dtype=torch.bfloat16)
    assert "qkv must be on a CUDA device" in err(lambda: lsk.qk_norm_rope(d, T, rows, None, None, 1e-6, A, A, A, A, A))
    assert "qkv must be bfloat16" in err(lambda: lsk.qk_norm_rope(d, T, rows.float(), None, None, 1e-6, A, A, A, A, A))
    assert "ws must be a tensor" in err(lambda: lsk.tree_attn(d, T, A, A, A, A, A, A, m, 0.1, A, A, A))
    p = torch.zeros(B, T, V)
    assert "probs must be float32" in err(lambda: lsk.verify_tree(d, T, p.half(), None, A, A, A, A, A, A, A, A))
    assert "probs must be a tensor" in err(lambda: lsk.verify_tree(d, T, A, None, A, A, A, A, A, A, A, A))
    assert "kmin" in err(lambda: lsk.make_cache_layers(d, None, None, None, None, None))
    assert "layers must be a table of Layer" in err(lambda: lsk.commit_path(d, T, (ctypes.c_int * 2)(), A, A, A, A, A, None))


def test_row_spacing():
    """Rows of [B, T, W] tensors may be slices of wider ones, evenly spaced; anything else is turned down."""
    from lookahead_sparse_kv_b200 import tree
    x = torch.zeros(3, 4, 20)
    bf = lambda t, rows, w: tree._rows(t, "call", "x", torch.float32, rows, w, t.get_device())  # noqa: E731
    assert bf(x, 12, 20)[1] == 20 and bf(x[..., :16], 12, 16)[1] == 20 and bf(x[:, :1, :16], 3, 16)[1] == 80
    assert bf(x[:1, :1, :16], 1, 16)[1] == 16 and bf(x.view(12, 20), 12, 20)[1] == 20
    for bad in (x[:, :3], x.transpose(0, 1), x[..., ::2], x.transpose(1, 2)):
        with pytest.raises(lsk.OasisError):
            bf(bad, bad.shape[0] * bad.shape[1], bad.shape[2])
    with pytest.raises(lsk.OasisError):
        bf(x, 11, 20)
    with pytest.raises(lsk.OasisError):
        bf(x, 12, 21)


def test_oracle_pins():
    """The fp64 statements on cases worked out by hand."""
    import numpy as np
    from oracle import tree_oracle as TO
    mask, pos = TO.tree_layout(np.array([[-1, 0, 0, 2]]), np.array([4]), np.array([10]))
    assert mask.tolist() == [[1, 3, 5, 13]] and pos.tolist() == [[10, 11, 11, 12]]
    p = np.array([[[0.5, 0.5, 0.0], [0.0, 0.25, 0.75]]])
    d = np.array([[[0.25, 0.75, 0.0], [1.0, 0.0, 0.0]]])
    one = lambda tok, ua, us: TO.verify_tree(p, d, np.array([[0, tok]]), np.array([[-1, 0]]), np.array([2]), np.array([[0, ua]]), np.array([us]))  # noqa: E731
    # token 1: stands below 0.5 / 0.75; else r = (0.25, 0, 0) and token 0 is drawn
    path, n, t = one(1, 0.6, 0.5)
    assert path.tolist() == [[0, 1]] and n.tolist() == [2] and t.tolist() == [2]
    path, n, t = one(1, 0.7, 0.9)
    assert path.tolist() == [[0, -1]] and n.tolist() == [1] and t.tolist() == [0]
    # token 0 is likelier to the target: it always stands; then 0.25 is the border of tokens 1 and 2
    assert one(0, 0.999, 0.25)[2].tolist() == [2] and one(0, 0.999, 0.2499)[2].tolist() == [1]
    q = np.zeros((1, 1, 1, 128))
    k = np.zeros((1, 1, 1, 16, 128))
    v = np.arange(16.0)[None, None, None, :, None] + k
    o, lse = TO.tree_attention(q, k, v, np.array([[[3]]]), np.array([3 * 16 + 4]), np.zeros((1, 1, 1, 128)), np.full((1, 1, 1, 128), 10.0),
                               np.array([[1]], np.uint64), 1.0)
    assert np.allclose(o, (0 + 1 + 2 + 3 + 10) / 5) and np.allclose(lse, np.log(5))
