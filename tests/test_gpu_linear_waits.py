"""Linear products whose waits run out on the GPU: reported, ended with nothing in flight, and followed by right ones.
Every wait of them has a limit; the products' results are not looked at."""
import pytest
import torch

from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    vsa_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vsa.load()


@pytest.fixture(autouse=True)
def _limits():
    yield
    assert vsa.load().vsa_linear_set_limits(1_000_000_000, 0) == 0
    vsa.linear_check()


def _randn(seed, *shape, std=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


# rows, K, F: fewer steps than stages of the ring; more; several tiles a pair; one CTA of the pair without rows
SHAPES = [(300, 128, 256), (300, 512, 256), (2000, 4096, 1024), (9000, 1024, 1536), (40, 4096, 512)]


@pytest.mark.parametrize("M,K,F", SHAPES)
def test_loads_that_come_after_the_limit(M, K, F):
    """One CTA of each pair asks for its operands when the MMAs have been given up; the product ends after them."""
    x, w, dy = _randn(1, 1, M, K), _randn(2, F, K), _randn(3, 1, M, F)
    L = vsa.load()
    ref = (vsa.linear(x, w), *vsa.linear_backward(x, w, dy)[:2])
    vsa.linear_check()
    calls = (lambda: vsa.linear(x, w), lambda: vsa.linear_backward(x, w, dy, want=(True, False)),
             lambda: vsa.linear_backward(x, w, dy, want=(False, True)))
    for call in calls:
        assert L.vsa_linear_set_limits(200_000, 2) == 0
        call()
        assert L.vsa_linear_set_limits(1_000_000_000, 0) == 0
        got = (vsa.linear(x, w), *vsa.linear_backward(x, w, dy)[:2])          # right behind it, on the same SMs
        with pytest.raises(vsa.VSAError, match="TIMEOUT"):
            vsa.linear_check()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("M,K,F", SHAPES)
def test_waits_of_next_to_no_time(M, K, F):
    """With a limit of a nanosecond any warp may give up anywhere, the epilogue's while MMAs run among them."""
    x, w, dy = _randn(1, 1, M, K), _randn(2, F, K), _randn(3, 1, M, F)
    L = vsa.load()
    ref = (vsa.linear(x, w), *vsa.linear_backward(x, w, dy)[:2])
    vsa.linear_check()
    for _ in range(5):
        assert L.vsa_linear_set_limits(1, 0) == 0
        vsa.linear(x, w)
        vsa.linear_backward(x, w, dy)
        assert L.vsa_linear_set_limits(1_000_000_000, 0) == 0
        got = (vsa.linear(x, w), *vsa.linear_backward(x, w, dy)[:2])
        try:
            vsa.linear_check()
        except vsa.VSAError as e:
            assert "TIMEOUT" in str(e)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
