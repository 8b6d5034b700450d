"""Feed-forward calls on the GPU where they are easily wrong: far arguments of
the activations, paths that only large calls take, shared and reused memory."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ffn_ref as ref
from gpu_util import banner
from test_gpu_ffn import KINDS, Experts, bnn, int8_rows, make, matrices, near, split  # noqa: F401 (bnn: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [1, 300])
@pytest.mark.parametrize("low,high", [(-115, -96), (-96, -88), (-88, -40), (-40, -20), (-20, -10), (-10, -5), (-5, 0), (0, 5), (5, 100)])
def test_silu_of_exact_arguments(bnn, P, low, high):
    """z = the bias, sums of 0.  Roundings, in half steps of fp32 (E32 of the value): exponential 2, its correction 1, product
    with z 1, sum 1, reciprocal 2, last product 1: 8.  Below the normal numbers the two products round to a
    step of their own, half of one each."""
    N = 1 << 16
    z = torch.from_numpy(np.random.default_rng(28).uniform(low, high, N).astype(np.float32)).cuda()
    W = bnn.ExpertWeights(torch.zeros((N, 4), dtype=torch.int32, device="cuda"), 16, alpha=torch.ones(1, device="cuda"), bias=z)
    banner(f"silu {P} {low} {high}")
    y = ref.f64(bnn.expert_linear(torch.zeros((P, 16), dtype=torch.int8, device="cuda"), W, act="silu"))
    want = ref.f64(z) / (1 + np.exp(-ref.f64(z)))
    off = np.abs(y - want) - 8 * ref.E32 * np.abs(want) - 2.0 ** -149
    assert off.max() <= 0, f"{(np.abs(y - want) / np.abs(want)).max() / ref.E32} half steps"


@pytest.mark.parametrize("P", [1, 300])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_activations_at_the_ends(bnn, P, act):
    """Infinite and very large arguments: the formulas' limits; -inf times 0 is NaN in them."""
    z = torch.tensor([np.inf, 3e38, 1e30, 161.0, 0.0, -0.0, -161.0, -1e13, -1e30, -3e38, -np.inf, np.nan], device="cuda")
    W = bnn.ExpertWeights(torch.zeros((12, 4), dtype=torch.int32, device="cuda"), 16, alpha=torch.ones(1, device="cuda"), bias=z)
    banner(f"ends {P} {act}")
    y = bnn.expert_linear(torch.zeros((P, 16), dtype=torch.int8, device="cuda"), W, act=act)[P - 1].cpu()
    assert torch.equal(y[:4], z[:4].cpu()) and (y[4:10] == 0).all() and torch.isnan(y[10:]).all()
