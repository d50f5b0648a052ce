"""commit_path where the path is not sound: what is written, what stays, and how far the context moves."""

import pytest
import torch

import lookahead_sparse_kv_b200 as lsk
from tests.test_gpu_tree import commit_case

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from lookahead_sparse_kv_b200 import build
    build.build()
    lsk.lib()
    yield
    assert lsk.read_device_error(clear=True) == 0


def test_bad_entries_take_their_positions_and_leave_them_as_they_were():
    """A block opened by bad entries alone, one opened by a bad entry before a sound one, a count above T over a padded path, one
    below 0: rows keep their places, skipped positions, slots and summaries stay, and each position taken counts."""
    T, N = 6, 4
    host, pool, st, kmin, kmax, k, v, path, count, c = commit_case(1, 4, 1, N, N, T, 3, [14, 16, 20, 33], [4, 3, 99, -2])
    path = torch.tensor([[0, 3, -1, 6, -1, -1], [9, 2, 4, -1, -1, -1], [1, 5, -1, -1, -1, -1], [0, 1, 2, 3, 4, 5]], dtype=I32)
    written = [(0, 14, 0), (0, 15, 3), (1, 17, 2), (1, 18, 4), (2, 20, 1), (2, 21, 5)]          # sequence, position, node
    want = {"host": host.clone(), "pool": pool.clone(), "kmin": kmin.clone(), "kmax": kmax.clone()}
    for b, pos, node in written:
        n, t = divmod(pos, 16)
        kr, vr = k[0, b, 0, node], v[0, b, 0, node]
        want["host"][0, b, 0, n, 0, t], want["host"][0, b, 0, n, 1, t] = kr, vr
        for s in (st[0, b, 0] == n).nonzero().flatten().tolist():
            want["pool"][0, b, 0, s, 0, t], want["pool"][0, b, 0, s, 1, t] = kr, vr
        first = t == 0 or (b, pos) == (1, 17)                                                   # the block's first sound row
        want["kmin"][0, b, 0, n] = kr if first else torch.minimum(want["kmin"][0, b, 0, n], kr)
        want["kmax"][0, b, 0, n] = kr if first else torch.maximum(want["kmax"][0, b, 0, n], kr)
    d = lsk.make_dims(4, 1, 1, N, N, 1, 0)
    pool, st, kmin, kmax, k, v = (t.to(DEV) for t in (pool, st, kmin, kmax, k, v))
    out = torch.empty(4, dtype=I32, device=DEV)
    lsk.commit_path(d, T, lsk.make_cache_layers(d, host, kmin, kmax, st, pool), k, v, path.to(DEV), count.to(DEV), c.to(DEV), out)
    assert lsk.read_device_error(clear=True) == lsk.DEVERR_ID_RANGE
    assert out.tolist() == [18, 19, 26, 33]
    for name, t in (("host", host), ("pool", pool), ("kmin", kmin), ("kmax", kmax)):
        assert torch.equal(t.cpu(), want[name]), name
