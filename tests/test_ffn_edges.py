"""The binding's checks of feed-forward calls, without a GPU: tensors that would
let a kernel past the caller's memory, or have it read other values."""
from __future__ import annotations

import pytest
import torch


@pytest.fixture
def on_host(monkeypatch):
    """Host tensors pass for device tensors; launches are recorded in `calls` and left out."""
    import xnor_popcount_gemm_amd as bnn
    bnn.lib()

    def dev(t, dtype, name):
        assert t.dtype is dtype, name
        return t

    calls = []
    monkeypatch.setattr(bnn, "_dev", dev)
    monkeypatch.setattr(bnn, "_on", lambda index, call, *args: calls.append(args) or 0)
    bnn.calls = calls
    yield bnn
    del bnn.calls


def planes_out(M, Xb):
    return {"Xb": Xb, "xsum": torch.zeros(M, dtype=torch.int32), "xscale": torch.zeros(M)}


@pytest.mark.parametrize("M", [1, 2, 5])
def test_planes_with_gaps_are_refused(on_host, M):
    """A row of planes is written up to its stride: a view of part of wider rows would have its neighbours overwritten, and
    the last one words past the end of its memory."""
    x = torch.zeros(M, 1000)
    big = torch.zeros(M, 8, 64, dtype=torch.int32)
    for view in (big[:, :, :32], big[:, :, 32:], big[:, :, 4:36]):
        with pytest.raises(ValueError, match="between its rows"):
            on_host.block_norm(x, out=planes_out(M, view))
    assert not on_host.calls
    on_host.block_norm(x, out=planes_out(M, big))
    on_host.block_norm(x, out=planes_out(M, torch.zeros(M, 8, 32, dtype=torch.int32)))
    assert len(on_host.calls) == 2


class Elsewhere(torch.Tensor):
    """A tensor that says it is on another device."""

    def get_device(self):
        return 1


def test_route_workspace_on_another_device_is_refused(on_host):
    """Its address goes to the kernel as it is."""
    logits = torch.zeros(100, 8)
    have = on_host.expert_route_workspace(100, 8, 2, device="cpu")
    with pytest.raises(ValueError, match="workspace"):
        on_host.expert_route(logits, 2, workspace=have.as_subclass(Elsewhere))
    with pytest.raises(ValueError, match="workspace"):
        on_host.expert_route(logits, 2, workspace=torch.zeros(2 * have.numel(), dtype=torch.uint8)[::2])
    assert not on_host.calls
    on_host.expert_route(logits, 2, workspace=have)
    on_host.expert_route(logits, 2)
    assert len(on_host.calls) == 2


@pytest.mark.parametrize("ternary", [False, True])
@pytest.mark.parametrize("E", [1, 3])
def test_planes_narrower_than_k_are_refused(on_host, E, ternary):
    """A view of a few words of wider rows has the stride of K but not its words."""
    wide = torch.zeros(E, 5, 16, dtype=torch.int32)
    alpha = torch.ones(E, 5)

    def lay_out(w, K):
        on_host.ExpertWeights(w, K, Zp=w if ternary else None, alpha=alpha)
    for view in (wide[:, :, :3], wide[:, :, 12:15], wide[:, :, 16:]):
        with pytest.raises(ValueError, match="words of K = 100"):
            lay_out(view, 100)
    assert not on_host.calls
    lay_out(wide[:, :, 12:], 100)
    lay_out(wide[:, :, :3], 96)
    lay_out(wide, 512)
    assert len(on_host.calls) == 3


def test_nonzero_plane_on_another_device_is_refused(on_host):
    S = torch.zeros(2, 5, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        on_host.ExpertWeights(S, 100, Zp=torch.zeros_like(S).as_subclass(Elsewhere), alpha=torch.ones(2))
    assert not on_host.calls
    on_host.ExpertWeights(S, 100, Zp=torch.zeros_like(S), alpha=torch.ones(2))


@pytest.mark.parametrize("E,N", [(2, 5), (7, 5), (4, 1), (3, 3)])
def test_scales_that_experts_share(on_host, E, N):
    """A row stride of 0 means one scale for each expert to the kernel, so the row is laid out for each of them."""
    S = torch.zeros(E, N, 4, dtype=torch.int32)
    row = torch.arange(1.0, N + 1)
    for alpha in (row.expand(E, N), row[:1].expand(E, N), row[:1, None].expand(E, N)):
        w = on_host.ExpertWeights(S, 100, alpha=alpha)
        address, stride = w._c[1:3]
        assert stride >= N and address == w.alpha.data_ptr() and w.alpha.is_contiguous() and torch.equal(w.alpha, alpha)
    own = torch.rand(E, N + 3)[:, :N]
    w = on_host.ExpertWeights(S, 100, alpha=own)      # rows with gaps are read where they are
    assert w._c[1:3] == (own.data_ptr(), N + 3)
    assert on_host.ExpertWeights(S, 100, alpha=torch.ones(E))._c[2] == 0


@pytest.mark.parametrize("name", ["W", "alpha", "bias"])
def test_weights_tensors_cannot_be_replaced(on_host, name):
    """The calls read them by the addresses that they had: another tensor in their place would leave those to be freed."""
    w = on_host.ExpertWeights(torch.zeros(2, 5, 4, dtype=torch.int32), 100, alpha=torch.ones(2, 5), bias=torch.zeros(2, 5))
    held = getattr(w, name)
    with pytest.raises(AttributeError):
        setattr(w, name, 2 * held)
    assert getattr(w, name) is held and held.data_ptr() in w._c


@pytest.mark.parametrize("E,N", [(2, 5), (4, 1)])
def test_biases_that_experts_share(on_host, E, N):
    """Laid out for each expert, as scales are; the C call refuses a stride of 0."""
    row = torch.arange(1.0, N + 1)
    w = on_host.ExpertWeights(torch.zeros(E, N, 4, dtype=torch.int32), 100, alpha=torch.ones(E), bias=row.expand(E, N))
    address, stride = w._c[3:5]
    assert stride >= N and address == w.bias.data_ptr() and torch.equal(w.bias, row.expand(E, N))
