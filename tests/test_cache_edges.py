"""The binding's checks of cache calls, without a GPU: shapes that would let a
kernel past the end of a tensor, and calls that have nothing to do."""
from __future__ import annotations

import ctypes
import random

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


def workspace_bytes(bnn, seqs, rows, nodes, ctx, heads, kv, dim):
    c, b = bnn._KvCache(), bnn._KvBatch()
    c.table, c.ld_table, c.num_pages, c.page_size, c.kv_heads, c.dim, c.dtype = 1 << 16, 4096, 1 << 20, 16, kv, dim, 1
    b.B, b.rows, b.max_nodes, b.max_ctx = seqs, rows, nodes, ctx
    return bnn.lib().bnn_tree_attention_workspace(ctypes.addressof(c), ctypes.addressof(b), heads)


@pytest.mark.parametrize("sizes", [
    # sequences, new tokens of each, committed tokens, heads, key heads, dim
    (64, 1, 2000, 32, 8, 128), (4, 1024, 8192, 32, 8, 128), (64, 64, 4000, 32, 8, 128), (1, 66, 60000, 1, 1, 128), (9, 17, 30000, 40, 5, 96),
    (3, 7, 65000, 16, 16, 256), (130, 33, 700, 12, 4, 64), (2, 2000, 500, 8, 1, 64)])
def test_attention_workspace_covers_smaller_calls(bnn, sizes):
    seqs, nodes, ctx, heads, kv, dim = sizes
    whole = workspace_bytes(bnn, seqs, seqs * nodes, nodes, ctx, heads, kv, dim)
    assert 0 < whole < 1 << 30
    rng = random.Random(repr(sizes))
    smaller = [(b, n, c) for b in {1, 2, seqs // 2 or 1, seqs} for n in {1, 2, 3, 16, 17, 33, nodes} if n <= nodes and b <= seqs for c in (ctx, ctx // 2, 100)]
    smaller += [(rng.randint(1, seqs), rng.randint(1, nodes), rng.randint(0, ctx)) for _ in range(300)]
    for b, n, c in smaller:
        if b <= seqs:
            for rows in {b * n, rng.randint(1, b * n)}:
                need = workspace_bytes(bnn, b, rows, n, c, heads, kv, dim)
                assert 0 <= need <= whole, (b, n, c, rows, need, whole)


def test_attention_refuses_more_rows_than_it_counts(bnn):
    assert workspace_bytes(bnn, 1, 1 << 25, 1 << 25, 10, 64, 1, 64) == -1       # 2^31 rows of one key head
    assert workspace_bytes(bnn, 1, 1 << 24, 1 << 24, 10, 64, 1, 64) >= 0
