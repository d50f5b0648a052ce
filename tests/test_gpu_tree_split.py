"""tree_attn's split of the work: CTAs that walk many segments (whole items, stretches cut after one tile, segments without a tile),
row-tile pairs beside single row tiles, and items joined from many parts.  Every row is compared with fp64 on the device.

Tolerance: a softmax weight is rounded to bf16, half a step 2^-8 of it, and the output once more: 2^-8 |o| + (2^-8 + 2^-16) A with A the
weighted mean of |v|; lse: fp32 scores, a few 2^-24 sum |q_c k_c|, here below 1e-4."""

import pytest
import torch

import lookahead_sparse_kv_b200 as lsk

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, I32 = torch.bfloat16, torch.int32
SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from lookahead_sparse_kv_b200 import build
    build.build()
    lsk.lib()
    yield
    assert lsk.read_device_error(clear=True) == 0


class Call:
    """One call's tensors.  kinds: per sequence "full" (random free slots), "free" (nothing resident) or "blind" (no row sees
    anything), taken in turn."""

    def __init__(self, B, T, hq, hkv, K, seed, kinds=("full",)):
        g = torch.Generator(DEV).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
        N = K + 3
        self.T, self.d = T, lsk.make_dims(B, hq, hkv, N, K, 1, 0)
        self.q, self.k, self.v = r(B, T, hq, 128), r(B, hkv, T, 128), r(B, hkv, T, 128)
        self.pool = r(B, hkv, K, 2, 16, 128)
        st = torch.rand(B, hkv, N, generator=g, device=DEV).argsort(-1)[..., :K]
        st = torch.where(torch.rand(B, hkv, K, generator=g, device=DEV) < 0.15, -1, st).int()
        self.ctx = (N * 16 - torch.randint(0, 40, (B,), generator=g, device=DEV)).int()
        up = torch.full((B, T), -1, dtype=I32, device=DEV)
        j = torch.arange(T, device=DEV)
        up[:] = torch.where(j > 0, (torch.rand(B, T, generator=g, device=DEV) * j).floor().int(), -1)
        self.mask, pos = torch.empty(B, T, dtype=torch.int64, device=DEV), torch.empty(B, T, dtype=I32, device=DEV)
        lsk.tree_layout(self.d, T, up, None, self.ctx, self.mask, pos)
        for b in range(B):
            if kinds[b % len(kinds)] == "free":
                st[b] = -1
            if kinds[b % len(kinds)] == "blind":
                self.mask[b] = 0
        self.st = st
        self.ws = torch.full((lsk.tree_workspace_bytes(self.d, T),), 255, dtype=torch.uint8, device=DEV)
        self.out, self.lse = torch.full((B, T, hq, 128), 9.0, dtype=BF, device=DEV), torch.full((B, T, hq), 9.0, device=DEV)

    def run(self, ws=None, stream=None):
        lsk.tree_attn(self.d, self.T, self.q, self.pool, self.st, self.ctx, self.k, self.v, self.mask, SCALE, self.out, self.lse,
                      self.ws if ws is None else ws, stream=stream)
        return self.out, self.lse

    def check(self):
        self.run()
        B, T, hq = self.lse.shape
        hkv, K = self.st.shape[1:]
        tok = torch.arange(16, device=DEV)
        valid = ((self.st[..., None] >= 0) & (self.st[..., None] * 16 + tok < self.ctx.view(B, 1, 1, 1))).flatten(2)
        sees = (self.mask[:, :, None] >> torch.arange(T, device=DEV) & 1).bool()
        for b in range(B):                                       # a sequence at a time: a few MB of doubles
            keys = torch.cat([self.pool[b, :, :, 0].flatten(1, 2), self.k[b]], 1).double()
            vals = torch.cat([self.pool[b, :, :, 1].flatten(1, 2), self.v[b]], 1).double()
            q = self.q[b].double().view(T, hkv, hq // hkv, 128).permute(1, 0, 2, 3)
            x = torch.einsum("htgc,hsc->htgs", q, keys) * SCALE
            on = torch.cat([valid[b, :, None].expand(-1, T, -1), sees[b].expand(hkv, -1, -1)], -1)
            on = on & sees[b].any(-1)[None, :, None]             # a row whose word is 0 sees nothing at all
            x = x.masked_fill(~on[:, :, None], float("-inf"))
            lse = torch.logsumexp(x, -1)
            w = torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[..., None])
            o, size = (torch.einsum("htgs,hsc->htgc", w, y) for y in (vals, vals.abs()))
            o, size = (y.permute(1, 0, 2, 3).reshape(T, hq, 128) for y in (o, size))
            lse = lse.permute(1, 0, 2).reshape(T, hq)
            over = (self.out[b].double() - o).abs() - (2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -16) * size + 1e-30)
            assert not bool((over > 0).any()), (b, over.max())
            fin = lse.isfinite()
            assert torch.equal(self.lse[b].isfinite(), fin) and bool((self.lse[b][~fin] == float("-inf")).all())
            assert float((self.lse[b].double() - lse)[fin].abs().max() if fin.any() else 0.0) <= 1e-4, b


@pytest.mark.parametrize("B,T,hq,hkv,K,kinds", [
    (200, 8, 8, 8, 8, ("free", "full", "blind", "free")),        # one tile, two or none, 13 items a CTA
    (64, 8, 8, 8, 5, ("full",)), (90, 3, 16, 8, 1, ("free", "free", "full")),
    (1, 7, 32, 8, 128, ("full",)),                               # stretches of two tiles over 17: cut after one
    (5, 8, 8, 8, 128, ("full", "free", "full", "blind", "full"))])
def test_segments_of_one_tile(B, T, hq, hkv, K, kinds):
    """One row tile and one KV tile: the second issuer has nothing to do in such a segment and may be any time late in it."""
    Call(B, T, hq, hkv, K, seed=B + K, kinds=kinds).check()


def test_a_gather_runs_beside_a_split_call():
    """The attention leaves SMs to a gather on another stream, and the kernel that joins the parts does not take them while it waits:
    a gather that gets ready early in the call ends well before it (1 MB against 0.8 GB; the median of nine)."""
    c = Call(12, 8, 64, 8, 1024, seed=2)
    g = torch.Generator().manual_seed(3)
    d = lsk.make_dims(1, 8, 8, 64, 64, 1, 16)
    host = torch.randn(1, 8, 64, 2, 16, 128, generator=g).to(BF).pin_memory()
    slot = torch.arange(16, dtype=I32, device=DEV).expand(1, 8, 16).contiguous()
    n, pool = torch.full((1, 8), 16, dtype=I32, device=DEV), torch.empty(1, 8, 64, 2, 16, 128, dtype=BF, device=DEV)
    copy = torch.cuda.Stream(priority=torch.cuda.Stream.priority_range()[1])
    share = []
    for i in range(12):
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        torch.cuda.synchronize()
        torch.cuda._sleep(200000)                                # both streams are filled before either starts
        ev[0].record()
        copy.wait_event(ev[0])
        with torch.cuda.stream(copy):
            torch.cuda._sleep(40000)                             # the call is under way
            lsk.prefetch(d, host, slot, slot, n, pool, stream=copy)
            ev[1].record(copy)
        c.run()
        ev[2].record()
        torch.cuda.synchronize()
        share.append(ev[0].elapsed_time(ev[1]) / ev[0].elapsed_time(ev[2]))
    assert torch.equal(pool[:, :, :16].cpu(), host[:, :, :16])
    assert sorted(share[3:])[4] < 0.9, share


@pytest.mark.parametrize("B,T,hq,hkv,K,kinds", [
    # (KV tiles a unit = K / 8 and the tree's; on 148 SMs, 132 CTAs)
    (64, 8, 8, 8, 24, ("full", "blind", "full", "free")),         # 512 items of 4 tiles: 4 whole ones a CTA
    (39, 8, 16, 8, 128, ("full", "full", "free", "blind", "full")),   # 312 of 17: stretches of 41 over up to 4 items
    (151, 40, 16, 2, 24, ("full", "free", "full")),               # pairs of row tiles, then single ones, whole
    (20, 40, 16, 2, 128, ("full", "full", "blind")),              # the same, cut
    (10, 64, 64, 8, 128, ("full", "free", "full", "full")),       # pairs alone, cut
    (100, 33, 12, 4, 9, ("blind", "full")), (25, 64, 8, 8, 100, ("full",))])
def test_many_segments_a_cta(B, T, hq, hkv, K, kinds):
    """Both list buffers come round several times, segments without a tile lie between full ones, and CTAs pass from items of two row
    tiles to items of one."""
    Call(B, T, hq, hkv, K, seed=B + T, kinds=kinds).check()


@pytest.mark.parametrize("T,hq", [(1, 1), (8, 4), (40, 16), (64, 16)])
def test_items_of_many_parts(T, hq):
    """One KV head over 1,024 slots: up to 65 parts to join, more than a warp has lanes."""
    Call(1, T, hq, 1, 1024, seed=T).check()


SPLIT = [(1, 7, 32, 8, 128), (2, 64, 16, 1, 1024)]


def bits(c):
    torch.cuda.synchronize()
    return c.out.view(torch.int16).clone(), c.lse.view(torch.int32).clone()


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("shape", SPLIT)
def test_split_calls_captured_on_one_workspace(shape):
    """Two graphs on one workspace, replayed in turn on other inputs: the eager calls' bits, whatever the workspace held."""
    first, second = Call(*shape, seed=1), Call(*shape, seed=2)
    want = []
    for c in (first, second):
        c.run()
        want.append(bits(c))
    a, b = Call(*shape, seed=3), Call(*shape, seed=4)
    graphs = []
    torch.cuda.synchronize()
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(ws=a.ws)
        graphs.append(g)
    for c, src in ((a, first), (b, second)):
        for n in ("q", "k", "v", "pool", "st", "ctx", "mask"):
            getattr(c, n).copy_(getattr(src, n))
    for _ in range(3):
        a.ws.fill_(255)
        for g in graphs:
            g.replay()
        assert same(bits(a), want[0]) and same(bits(b), want[1])


@pytest.mark.parametrize("shape", SPLIT)
def test_split_calls_on_two_streams(shape):
    """Two calls at once, each with a workspace of its own, give what each gives alone; so do calls that follow one another closely."""
    both = [Call(*shape, seed=s) for s in (5, 6)]
    want = []
    for c in both:
        c.run()
        want.append(bits(c))
        c.out.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(both, streams):
            c.run(stream=s)
    assert all(same(bits(c), w) for c, w in zip(both, want))
    for _ in range(10):                                          # one stream, one workspace: the next call waits for the join
        for c in both:
            c.run(ws=both[0].ws)
    assert all(same(bits(c), w) for c, w in zip(both, want))


@pytest.mark.parametrize("shape", SPLIT)
def test_split_calls_write_only_their_buffers(shape):
    """Guard bands around a workspace of exactly the size asked for, and around the outputs."""
    c = Call(*shape, seed=7)
    c.run()
    want = bits(c)
    raw = {}
    for n in ("ws", "out", "lse"):
        t = getattr(c, n)
        size = t.numel() * t.element_size()
        raw[n] = torch.full((size + 2048,), 0xA5, dtype=torch.uint8, device=DEV)
        setattr(c, n, raw[n][1024:1024 + size].view(t.dtype).view(t.shape))
    inputs = [getattr(c, n) for n in ("q", "k", "v", "pool", "st", "ctx", "mask")]
    kept = [t.clone() for t in inputs]
    c.run()
    assert same(bits(c), want)
    for n, t in raw.items():
        assert bool((t[:1024] == 0xA5).all()) and bool((t[-1024:] == 0xA5).all()), n
    assert bool((raw["ws"][1024:-1024] != 0xA5).any())           # the parts went there
    assert all(torch.equal(a, b) for a, b in zip(inputs, kept))
