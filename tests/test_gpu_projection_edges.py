"""Calls of the projection side that its documentation allows at the edges of their arguments."""
import pytest
import torch

from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    vsa_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vsa.load()


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    vsa.linear_check()


def _randn(seed, *shape, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _odd(x, stride):
    """x with another stride in its dimensions of length 1, which no address may come from."""
    return x.as_strided(x.shape, [stride if n == 1 else s for n, s in zip(x.shape, x.stride())])


@pytest.mark.parametrize("stride", [1, 3, 2 ** 33 + 5])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 70), (2, 1, 33), (2, 3, 1), (1, 5, 1)], ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_strides_of_dimensions_of_length_one(dtype, shape, stride):
    B, h, N = shape
    q, k, dq, dk = (_randn(i, B, n, N, 64, dtype=dtype) for i, n in enumerate((h, 1, h, 1)))
    odd = [_odd(t, stride) for t in (q, k, dq, dk)]
    w = _randn(9, 64, dtype=torch.float32)
    rot = vsa.Rotation(64, (24, 20, 20))
    kw = dict(grid=(1, 1, N))
    for fn in (vsa.rope, vsa.rope_backward):
        ref, got = fn(q, k, rot, **kw), fn(odd[0], odd[1], rot, **kw)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    ref, got = (vsa.qk_norm_rope(*a, w, None, rot, **kw) for a in ((q, k), odd[:2]))
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    ref = vsa.qk_norm_rope_backward(q, k, w, w, dq, dk, rot, **kw)
    got = vsa.qk_norm_rope_backward(odd[0], odd[1], w, w, odd[2], odd[3], rot, **kw)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    out = [torch.empty_like(q), torch.empty_like(k)]
    vsa.rope(q, k, rot, q_out=_odd(out[0], stride), k_out=_odd(out[1], stride), **kw)
    assert all(torch.equal(a, b) for a, b in zip(out, vsa.rope(q, k, rot, **kw)))
    if dtype != torch.float32:
        weight = _randn(10, 72, h * 64, dtype=dtype)
        assert torch.equal(vsa.linear(odd[0], weight), vsa.linear(q, weight))
        g = _randn(11, B, N, 72, dtype=dtype)
        got, ref = (vsa.linear_backward(x, weight, d, bias=True) for x, d in ((odd[0], _odd(g, stride)), (q, g)))
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
