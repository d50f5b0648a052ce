"""make_cache_layers takes tensors stacked over layers without a gap: a stack of larger layers has its layers elsewhere than the table
would say, and is turned down.  CPU only."""

import pytest
import torch

import lookahead_sparse_kv_b200 as lsk
from lookahead_sparse_kv_b200 import build as lsk_build

BF = torch.bfloat16
L, B, H, N, K = 3, 2, 2, 8, 4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lsk_build.build()


def tensors(n=N, k=K, layers=L):
    z = lambda *s, t=BF: torch.zeros(layers, B, H, *s, dtype=t)  # noqa: E731
    return {"host_kv": z(n, 2, 16, 128), "kmin": z(n, 128), "kmax": z(n, 128), "slot_table": z(k, t=torch.int32), "pool": z(k, 2, 16, 128)}


def call(name, x):
    """What the call says of `x` in place of the sound tensor (on the CPU, where a sound one is turned down for its device alone)."""
    from lookahead_sparse_kv_b200 import tree
    sound = tensors()
    each = sound[name].numel() // L
    with pytest.raises(lsk.OasisError) as e:
        tree._stack(x, "make_cache_layers", name, x.dtype, L, each, 0)
    assert e.value.code == lsk.EINVAL
    return str(e.value)


@pytest.mark.parametrize("name", ["host_kv", "kmin", "kmax", "slot_table", "pool"])
def test_layers_of_another_size_are_turned_down(name):
    assert "elements a layer" in call(name, tensors(n=N + 2, k=K + 1)[name])
    assert "elements a layer" in call(name, tensors(n=N + 2, k=K + 1, layers=L + 1)[name])
    assert "must be on a CUDA device" in call(name, tensors()[name])
    assert "must be on a CUDA device" in call(name, tensors(layers=L + 2)[name])        # more layers than are used
    assert "must be on a CUDA device" in call(name, tensors()[name].flatten())
    assert "the call needs" in call(name, tensors(layers=L - 1)[name])


def test_the_call_itself():
    d = lsk.make_dims(B, H, H, N, K, 1, 0)
    t = tensors(n=N + 2)
    with pytest.raises(lsk.OasisError) as e:
        lsk.make_cache_layers(d, None, t["kmin"], t["kmax"], None, None)
    assert "kmin must hold" in str(e.value)
