"""The draft-tree calls at the ends of what they take: nothing written outside the buffers, offsets beyond 32 bits, host memory that
the device cannot address, a batch whose every tree is empty."""

import numpy as np
import pytest
import torch

import lookahead_sparse_kv_b200 as lsk
from tests.test_gpu_tree_step import B, HKV, HQ, K, N, RESULTS, one_step, step_tensors

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


def guarded(t):
    """A copy of t between two bands of 64 marked elements, and a check that the bands are as they were."""
    flat = torch.zeros(t.numel() + 128, dtype=t.dtype, device=t.device, pin_memory=not t.is_cuda)
    raw = flat.view(torch.uint8)
    raw.fill_(0xA5)
    view = flat[64:64 + t.numel()].view(t.shape)
    view.copy_(t)
    size, n = t.element_size(), t.numel()
    return view, lambda: bool((raw[:64 * size] == 0xA5).all()) and bool((raw[(64 + n) * size:] == 0xA5).all())


@pytest.mark.parametrize("T", [1, 5, 33, 64])
def test_nothing_is_written_outside_the_buffers(T):
    d = lsk.make_dims(B, HQ, HKV, N, K, 1, 0)
    plain, s = step_tensors(d, T, 7), step_tensors(d, T, 7)
    checks = {}
    for n in [*RESULTS, "ws"]:
        s[n], checks[n] = guarded(s[n])
    s["layers"] = lsk.make_cache_layers(d, s["host"], s["kmin"], s["kmax"], s["st"], s["pool"])
    keep = {n: s[n].clone() for n in s if isinstance(s[n], torch.Tensor) and n not in RESULTS and n != "ws"}
    one_step(d, T, plain)
    one_step(d, T, s)
    torch.cuda.synchronize()
    for n, ok in checks.items():
        assert ok(), n
    for n in RESULTS:
        a, b = (x.view(torch.int64) if x.dtype == torch.uint64 else x for x in (plain[n], s[n]))
        assert torch.equal(a, b), n
    for n, t in keep.items():
        assert torch.equal(s[n], t), f"input {n} was changed"


def test_a_batch_of_empty_trees():
    """No real node anywhere: nothing stands, nothing is committed, every attention row is empty."""
    T = 6
    d = lsk.make_dims(B, HQ, HKV, N, K, 1, 0)
    s = step_tensors(d, T, 9)
    s["n"].zero_()
    kept = {n: s[n].clone() for n in ("host", "pool", "kmin", "kmax")}
    one_step(d, T, s)
    torch.cuda.synchronize()
    assert not s["out"].any() and (s["lse"] == float("-inf")).all()
    assert not s["cnt"].any() and (s["next"] == -1).all() and (s["path"] == -1).all() and torch.equal(s["ctx_out"], s["ctx"])
    for n, t in kept.items():
        assert torch.equal(s[n], t), n


def test_projection_rows_far_apart():
    """Six rows 2^29 elements apart: offsets beyond 2^31."""
    hq, hkv, step = 2, 1, 1 << 29
    d = lsk.make_dims(2, hq, hkv, 64, 16, 1, 0)
    flat = torch.empty(5 * step + 512, dtype=BF, device=DEV)
    qkv = flat.as_strided((2, 3, 512), (3 * step, step, 1))
    rows = torch.randn(2, 3, 512, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    qkv.copy_(rows)
    inv, pos = torch.ones(64, device=DEV), torch.arange(6, dtype=I32, device=DEV).view(2, 3)
    got, want = ([torch.empty(s, dtype=BF, device=DEV) for s in ((2, 3, 2, 128), (2, 1, 3, 128), (2, 1, 3, 128))] for _ in range(2))
    lsk.qk_norm_rope(d, 3, qkv, None, None, 1e-6, inv, pos, *got)
    lsk.qk_norm_rope(d, 3, rows, None, None, 1e-6, inv, pos, *want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_probability_rows_far_apart():
    """Six rows 2^29 + 1 floats apart (offsets beyond 2^31, each row at another alignment) against the same rows packed."""
    V, step = 50001, (1 << 29) + 1
    d = lsk.make_dims(2, 1, 1, 64, 16, 1, 0)
    g = torch.Generator().manual_seed(2)
    flat = torch.empty(5 * step + V, device=DEV)
    far = flat.as_strided((2, 3, V), (3 * step, step, 1))
    rows = torch.softmax(3 * torch.randn(2, 3, V, generator=g), -1).to(DEV)
    far.copy_(rows)
    tok, par = torch.randint(0, V, (2, 3), generator=g).int().to(DEV), torch.tensor([[-1, 0, 1]] * 2, dtype=I32, device=DEV)
    outs = []
    for p in (far, rows):
        for u in (0.0, 0.7):                       # every draft stands, or none
            o = [torch.empty(2, 3, dtype=I32, device=DEV), torch.empty(2, dtype=I32, device=DEV), torch.empty(2, dtype=I32, device=DEV)]
            lsk.verify_tree(d, 3, p, None, tok, par, None, torch.full((2, 3), u, device=DEV), torch.tensor([0.3, 0.8], device=DEV), *o)
            outs.append([t.tolist() for t in o])
    assert outs[:2] == outs[2:] and outs[0][1] == [3, 3] and outs[1][1] == [1, 1]


def test_pool_beyond_four_gigabytes():
    """The last unit of a 4.8-GB pool, budget 1024, against fp64 on the device."""
    Bb, H, Kb, T = 72, 8, 1024, 3
    d = lsk.make_dims(Bb, H, H, 1024, Kb, 1, 0)
    g = torch.Generator(DEV).manual_seed(3)
    pool = torch.empty(Bb, H, Kb, 2, 16, 128, dtype=BF, device=DEV)
    pool[:-1].zero_()
    pool[-1] = torch.randn(H, Kb, 2, 16, 128, generator=g, device=DEV).to(BF)
    st = torch.arange(Kb, dtype=I32, device=DEV).expand(Bb, H, Kb).contiguous()
    ctx = torch.full((Bb,), Kb * 16 - 7, dtype=I32, device=DEV)
    q, k, v = (torch.randn(s, generator=g, device=DEV).to(BF) for s in ((Bb, T, H, 128), (Bb, H, T, 128), (Bb, H, T, 128)))
    mask = torch.tensor([1, 3, 5], device=DEV).expand(Bb, T).contiguous()
    out, lse = torch.empty(Bb, T, H, 128, dtype=BF, device=DEV), torch.empty(Bb, T, H, device=DEV)
    ws = torch.empty(lsk.tree_workspace_bytes(d, T), dtype=torch.uint8, device=DEV)
    lsk.tree_attn(d, T, q, pool, st, ctx, k, v, mask, 128 ** -0.5, out, lse, ws)
    for h in (0, H - 1):
        keys = torch.cat([pool[-1, h, :, 0].reshape(-1, 128)[:-7], k[-1, h]]).double()
        vals = torch.cat([pool[-1, h, :, 1].reshape(-1, 128)[:-7], v[-1, h]]).double()
        x = q[-1, :, h].double() @ keys.T * 128 ** -0.5
        sees = mask[-1, :, None] >> torch.arange(T, device=DEV) & 1
        x[:, -T:] = torch.where(sees.bool(), x[:, -T:], float("-inf"))
        w = torch.softmax(x, -1)
        ref, size = w @ vals, w @ vals.abs()
        # bf16 weights and a bf16 store: 2^-8 |o| + (2^-8 + 2^-16) A
        over = (out[-1, :, h].double() - ref).abs() - (2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -16) * size)
        assert not bool((over > 0).any())
        assert float((lse[-1, :, h].double() - torch.logsumexp(x, -1)).abs().max()) <= 1e-4


def test_host_memory_that_is_not_mapped_is_turned_down():
    d = lsk.make_dims(B, HQ, HKV, N, K, 1, 0)
    s = step_tensors(d, 4, 5)
    layers = lsk.make_cache_layers(d, torch.zeros(s["host"].shape, dtype=BF), s["kmin"], s["kmax"], s["st"], s["pool"])
    with pytest.raises(lsk.OasisError) as e:
        lsk.commit_path(d, 4, layers, s["k"], s["v"], s["path"], s["cnt"], s["ctx"], s["ctx_out"])
    assert e.value.code == lsk.ENOTMAPPED
    with pytest.raises(lsk.OasisError):
        lsk.make_cache_layers(d, s["host"].to(DEV), s["kmin"], s["kmax"], s["st"], s["pool"])


def test_long_and_repeated_calls_are_repeatable():
    """The same call gives the same bits: parts are joined in a fixed order."""
    d = lsk.make_dims(1, 16, 2, 400, 300, 1, 0)
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)  # noqa: E731
    T = 40
    q, pool, k, v = r(1, T, 16, 128), r(1, 2, 300, 2, 16, 128), r(1, 2, T, 128), r(1, 2, T, 128)
    st = torch.arange(300, dtype=I32, device=DEV).expand(1, 2, 300).contiguous()
    ctx = torch.tensor([4795], dtype=I32, device=DEV)
    mask = torch.full((1, T), (1 << T) - 1, device=DEV)
    ws = torch.empty(lsk.tree_workspace_bytes(d, T), dtype=torch.uint8, device=DEV)
    seen = []
    for _ in range(6):
        out, lse = torch.empty(1, T, 16, 128, dtype=BF, device=DEV), torch.empty(1, T, 16, device=DEV)
        lsk.tree_attn(d, T, q, pool, st, ctx, k, v, mask, 0.1, out, lse, ws)
        seen.append((out, lse))
    assert all(torch.equal(a, seen[0][0]) and torch.equal(b, seen[0][1]) for a, b in seen)
