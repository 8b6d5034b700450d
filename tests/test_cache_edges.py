"""The binding's checks of cache calls, without a GPU: shapes that would let a
kernel past the end of a tensor, and calls that have nothing to do."""
from __future__ import annotations

import pytest
import torch


@pytest.fixture(scope="module")
def bnn():
    import xnor_popcount_gemm_amd as m
    m.lib()
    return m


@pytest.fixture
def on_host(bnn, monkeypatch):
    """Host tensors pass for device tensors: shapes are looked at, nothing is launched."""
    def dev(t, dtype, name):
        assert t.dtype is dtype, name
        return t
    monkeypatch.setattr(bnn, "_dev", dev)
    return bnn


def cache(bnn, pages=8, table=None, pos=None, score=None):
    k = torch.zeros(pages, 4, 2, 64, dtype=torch.bfloat16)
    return bnn.KVCache(k, k.clone(), table, pos=None if pos is None else torch.zeros(pos, dtype=torch.int32),
                       score=None if score is None else torch.zeros(score))


def test_slot_tensors_have_a_row_for_each_sequence(on_host):
    table = torch.zeros(8, 3, dtype=torch.int32)
    assert cache(on_host, table=table, pos=(8, 2, 12), score=(9, 2, 13)).sequences == 8
    for bad in (dict(pos=(1, 2, 12)), dict(score=(7, 2, 12)), dict(pos=(8, 2, 12), score=(1, 2, 12)), dict(pos=(0, 2, 12))):
        with pytest.raises(ValueError, match="8 sequences"):
            cache(on_host, table=table, **bad)
    for bad in (dict(pos=(8, 1, 12)), dict(score=(8, 2, 11)), dict(pos=(8, 24))):
        with pytest.raises(ValueError, match="contiguous"):
            cache(on_host, table=table, **bad)


def test_slot_tensors_bound_the_sequences_without_a_table(on_host):
    assert cache(on_host).sequences == 8
    assert cache(on_host, pos=(3, 2, 4)).sequences == 3 and cache(on_host, pos=(8, 2, 4), score=(2, 2, 4)).sequences == 2

    class Device(torch.Tensor):   # a host tensor that says it is the GPU's
        is_cuda = True

    ints = lambda n: torch.zeros(n, dtype=torch.int32).as_subclass(Device)
    c = cache(on_host, score=(2, 2, 4))
    assert on_host._batch(c, ints(3), ints(2), 2, 1, 4)
    with pytest.raises(ValueError, match="at most the cache's sequences"):
        on_host._batch(c, ints(4), ints(3), 3, 1, 4)
