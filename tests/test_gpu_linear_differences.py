"""Gradients of the linear product against differences, each along directions of its own.

The loss is the fp64 formula. Each gradient's sum along a direction e of one input may be off by what the roundings
make, which are independent of one another:
  dx, dW   half a step of bf16 (2^-8) of each entry
  z        half a step, which changes act' by at most 1.2 of it (|act''| of silu, gelu and its tanh form is below 1.13)
  dz       half a step of it
so a sum with errors of at most s_i has a standard deviation of at most s = sqrt(sum s_i^2 / 3) where they are
uniform; six of them, and half of a hundredth for fp32 sums and the difference, are the tolerance.
"""
import pytest
import torch

import test_gpu_linear as tl
from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    vsa_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vsa.load()


@pytest.mark.parametrize("N", [7, 150])
@pytest.mark.parametrize("act", [None, "silu", "gelu", "gelu_tanh"])
def test_each_gradient_matches_differences(act, N):
    K, F, half = 256, 136, 2.0 ** -8
    x, w = tl._randn(1, 2, N, K, dtype=torch.bfloat16), tl._randn(2, F, K, dtype=torch.bfloat16, std=0.06)
    b, g = tl._randn(3, F, dtype=torch.float32), tl._randn(4, 2, N, F, dtype=torch.bfloat16)
    z = torch.empty(2, N, F, dtype=torch.bfloat16, device="cuda")
    vsa.linear(x, w, b, activation=act, z=z)
    grads = vsa.linear_backward(x, w, g, z=z if act else None, activation=act, bias=True)
    inputs, g64 = [t.double() for t in (x, w, b)], g.double()

    def loss(which, e, h):
        x, w, b = (t + h * e if i == which else t for i, t in enumerate(inputs))
        return (tl._act(x @ w.t() + b, act) * g64).sum()

    z64 = inputs[0] @ inputs[1].t() + inputs[2]
    off_z = 1.2 * half * z64.abs() * g64.abs() if act else torch.zeros_like(z64)
    dz = g64 * (tl._slope(z64, act) if act else 1.0)
    off_dz = off_z + (half * dz.abs() if act else 0.0)
    for which, (name, grad) in enumerate(zip(("dx", "dw", "db"), grads)):
        slopes, tols = [], []
        for seed in range(4):
            e = tl._randn(10 + seed, *grad.shape, dtype=torch.float64)
            slope = (loss(which, e, 1e-4) - loss(which, e, -1e-4)) / 2e-4
            got = (grad.double() * e).sum()
            own = (half * grad.double() * e).flatten() if which < 2 else torch.zeros(1, dtype=torch.float64, device="cuda")
            dual = e @ inputs[1].t() if which == 0 else inputs[0] @ e.t() if which == 1 else e.expand_as(z64)
            via = ((off_dz if which < 2 else off_z) * dual).flatten()
            tol = 6 * ((own.square().sum() + via.square().sum()) / 3).sqrt() + 5e-3 * grad.double().norm()
            assert abs(slope - got) <= tol, (name, seed, slope.item(), got.item(), tol.item())
            slopes.append(abs(slope).item())
            tols.append(tol.item())
        # without the gradient, with its opposite, or with a fifth too little of it, one of the directions fails
        assert max(s / t for s, t in zip(slopes, tols)) > 5, (name, slopes, tols)
