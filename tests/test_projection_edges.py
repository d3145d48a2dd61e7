"""CPU checks of the projection side's arguments at their edges."""
import ctypes

import pytest

from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa


@pytest.fixture(scope="module")
def lib():
    vsa_build.build()
    return vsa.load()


def _rope(lib, N=4, rot=None, positions=None, **kw):
    """vsa_rope on made-up addresses, which no refused or empty call touches."""
    sizes = vsa.RopeSizes(0, 1, N, 64)
    rot = rot or vsa.Rotation(64, (24, 20, 20)).spec
    positions = positions or vsa.Positions(kw.get("T", 1), kw.get("H", 1), kw.get("W", N))
    t = vsa.Heads(1 << 20, 1, 64 * N, 64 * N, 64)
    o = vsa.Heads(1 << 24, 1, 64 * N, 64 * N, 64)
    return lib.vsa_rope(ctypes.byref(sizes), ctypes.byref(rot), ctypes.byref(positions), ctypes.byref(t), None,
                        ctypes.byref(o), None, None)


@pytest.mark.parametrize("freq", [2.0 ** 64, -2.0 ** 64, 1e300, float("inf"), float("nan")])
def test_refusals_of_frequencies(lib, freq):
    rot = vsa.Rotation(64, (24, 20, 20)).spec
    rot.freq[3] = freq
    assert _rope(lib, rot=rot) == 1
    rot.freq[3] = 2.0 ** 63
    assert _rope(lib, N=0, rot=rot, positions=vsa.Positions(list=1 << 20)) == 0


@pytest.mark.parametrize("T,H,W", [(0, 4, 4), (2, 0, 3), (2, 3, 0), (0, 0, 0)])
def test_a_grid_without_tokens(lib, T, H, W):
    assert _rope(lib, N=0, T=T, H=H, W=W) == 0
    assert _rope(lib, N=1, T=T, H=H, W=W) == 2
    assert _rope(lib, N=0, T=T, H=H, W=-1) == 2
