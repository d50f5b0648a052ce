"""verify_tree over large vocabularies, on both sides of the choice between 8 and 16 CTAs a sequence (16 for few sequences over more
than 65,536 entries), against the fp64 statement: path, count and token are equal."""

import numpy as np
import pytest
import torch

import lookahead_sparse_kv_b200 as lsk
from oracle import tree_oracle as TO
from tests.test_gpu_tree import run_verify, verify_inputs

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from lookahead_sparse_kv_b200 import build
    build.build()
    lsk.lib()
    yield
    assert lsk.read_device_error(clear=True) == 0


def matches(p, q, tok, par, n, ua, us, V):
    ref = TO.verify_tree(p[..., :V].numpy(), None if q is None else q[..., :V].numpy(), tok.numpy(), par.numpy(), n.numpy(), ua.numpy(),
                         us.numpy())
    got = run_verify(p, q, tok, par, n, ua, us, V)
    for x, y in zip(got, ref):
        assert np.array_equal(x, y), (x, y)
    return ref


@pytest.mark.parametrize("B,T,V,shape,pad", [(1, 6, 70001, "star", 0), (9, 4, 70001, "tree", 3), (10, 4, 70001, "tree", 0),
                                             (1, 5, 65536, "star", 1), (1, 5, 65537, "star", 0), (2, 7, 151669, "tree", 2),
                                             (1, 26, 128256, "tree", 0)])
@pytest.mark.parametrize("draft", [True, False])
def test_large_vocabularies(B, T, V, shape, pad, draft):
    g = torch.Generator().manual_seed(B * T + V)
    some = 0
    for k in range(3):
        p, q, tok, par, n, ua, us = verify_inputs(B, T, V, g, shape, pad, noise=1.0 + k, ragged=B > 2)
        ref = matches(p, q if draft else None, tok, par, n, ua, us, V)
        some += int((ref[1] > 0).sum())
    assert some > 0


@pytest.mark.parametrize("draft", [True, False])
def test_draws_from_either_end_and_entries_that_are_no_probabilities(draft):
    """The draw falls into the first and into the last CTA's share; infinities, NaN, negative and subnormal entries on the way."""
    B, T, V = 4, 5, 99991
    g = torch.Generator().manual_seed(5)
    p, q, tok, par, n, ua, us = verify_inputs(B, T, V, g, "star", 0, noise=2.0, ragged=False)
    us = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5, 1e-6])
    for k, x in enumerate((float("inf"), float("-inf"), float("nan"), -0.25, -0.0, 1e-42)):
        for t in (p, q):
            t.scatter_(2, torch.randint(0, V, (B, T, 7), generator=g), x)
    ref = matches(p, q if draft else None, tok, par, n, ua, us, V)
    assert ref[2][0] < V // 16 and ref[2][1] > V - V // 16
    p[1, :, -V // 16:], p[1, :, -1] = 0.0, 1.0                      # nothing but the very last entry there
    assert matches(p, q if draft else None, tok, par, n, torch.full((B, T), 0.9999), us, V)[2][1] == V - 1


def test_nothing_left_and_no_mass():
    """A target equal to its draft that is turned down all the same (a zero there) leaves nothing: drawn from the row itself; a row
    without mass: -1."""
    V = 80001
    p = torch.zeros(2, 3, V)
    p[0, 0, 77777], p[0, 0, 5] = 0.5, 0.5
    q = p.clone()
    q[0, 0, 9] = 0.25
    tok = torch.tensor([[0, 9, 9], [0, 1, 2]], dtype=I32)
    par = torch.tensor([[-1, 0, 0]] * 2, dtype=I32)
    n = torch.full((2,), 3, dtype=I32)
    ref = matches(p, q, tok, par, n, torch.zeros(2, 3), torch.tensor([0.75, 0.5]), V)
    assert ref[1].tolist() == [1, 1] and ref[2].tolist() == [77777, -1]
